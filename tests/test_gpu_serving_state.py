"""What the binding keeps between the serving calls: descriptions of a cache and
a batch, and the attention's workspaces."""
import threading

import pytest
import torch

from test_gpu_serving import full_cache, gen, make_batch, tensors, values

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    from bit_error_compensated_gb300 import echo
    echo.echo_serving_status()


# ------------------------------------------------- caches and batches that change
def largest(g, n=6, length=40, page=16):
    starts, table, pages = make_batch([1] * n, [length + i for i in range(n)], page, g)
    cache = full_cache(g, pages, page, 2, 64, 8)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")           # noqa: E731
    return cache, ints(starts), ints([length + i for i in range(n)]), table


def attend(cache, batch, q):
    from bit_error_compensated_gb300 import echo
    out = torch.full_like(q, 7)
    echo.echo_attention(cache, batch, q, out)
    return out


@pytest.mark.parametrize("how", ["assigned", "resized"])
def test_a_smaller_batch_in_the_same_memory(how):
    """A server keeps arrays of its largest batch and takes their first n: the
    addresses stay, the sequences that are gone are neither written nor attended."""
    from bit_error_compensated_gb300 import echo
    g = gen(1)
    cache, starts, lengths, table = largest(g)
    batch = echo.CacheBatch(starts[:], lengths[:], table[:])
    q = values(g, 6, 4, 64, dtype=torch.bfloat16)
    k, v = values(g, 6, 2, 64), values(g, 6, 2, 64)
    before = cache.codes.clone()
    echo.echo_cache_append(cache, batch, k, v)
    full = attend(cache, batch, q)
    cache.codes.copy_(before)
    want_cache = echo.Cache(cache.pages, 16, 2, 64, 8, codes=before.clone(), meta=cache.meta.clone())
    fresh = echo.CacheBatch(starts[:3].clone(), lengths[:2].clone(), table[:2].clone())
    echo.echo_cache_append(want_cache, fresh, k, v)
    if how == "assigned":
        batch.starts, batch.lengths, batch.table = starts[:3], lengths[:2], table[:2]
    else:
        batch.starts.resize_(3), batch.lengths.resize_(2), batch.table.resize_(2, table.shape[1])
    echo.echo_cache_append(cache, batch, k, v)
    assert torch.equal(cache.codes, want_cache.codes)
    out = attend(cache, batch, q)
    assert torch.all(out[2:] == 7) and torch.equal(out[:2], attend(want_cache, fresh, q)[:2])
    assert not torch.equal(full[2:], out[2:])
    assert echo.echo_serving_status() == 0


def test_a_table_of_another_stride_in_the_same_memory():
    from bit_error_compensated_gb300 import echo
    g = gen(2)
    cache, starts, lengths, table = largest(g)
    wide = torch.full((6, 2 * table.shape[1]), -1, dtype=torch.int32, device="cuda")
    wide.view(-1)[:table.numel()] = table.flatten()
    batch = echo.CacheBatch(starts, lengths, wide.view(-1)[:table.numel()].view_as(table))
    q = values(g, 6, 4, 64, dtype=torch.bfloat16)
    want = attend(cache, batch, q)
    wide.fill_(-1)
    wide[:, :table.shape[1]] = table
    batch.table = wide[:, :table.shape[1]]
    assert torch.equal(attend(cache, batch, q), want)
    wide.view(-1)[:table.numel()] = table.flatten()
    batch.table.data = wide.view(-1)[:table.numel()].view_as(table)
    assert torch.equal(attend(cache, batch, q), want)
    assert echo.echo_serving_status() == 0


def test_arrays_that_no_longer_fit_are_refused():
    from bit_error_compensated_gb300 import echo
    g = gen(3)
    cache, starts, lengths, table = largest(g)
    batch = echo.CacheBatch(starts, lengths, table)
    q = values(g, 6, 4, 64, dtype=torch.bfloat16)
    attend(cache, batch, q)
    batch.lengths = lengths[:4]                              # of six sequences
    for _ in range(2):
        with pytest.raises(ValueError, match="lengths"):
            attend(cache, batch, q)
    batch.lengths = lengths
    batch.starts = starts.view(torch.float32)
    with pytest.raises(ValueError, match="starts"):
        attend(cache, batch, q)
    batch.starts = starts
    attend(cache, batch, q)


def test_a_cache_whose_tensors_change_is_checked_again():
    from bit_error_compensated_gb300 import echo
    g = gen(4)
    cache, starts, lengths, table = largest(g)
    batch = echo.CacheBatch(starts, lengths, table)
    q = values(g, 6, 4, 64, dtype=torch.bfloat16)
    want = attend(cache, batch, q)
    whole = cache.codes, cache.meta
    cache.codes = whole[0][:3]                               # the same address, fewer pages
    with pytest.raises(ValueError, match="codes"):
        attend(cache, batch, q)
    cache.codes, cache.pages, cache.meta = whole[0][:3], 3, whole[1][:3]
    attend(cache, batch, q)                                  # pages past the third are not there
    assert echo.echo_serving_status() == echo.ECHO_ERR_ARG
    cache.codes, cache.pages, cache.meta = whole[0], len(whole[1]), whole[1]
    assert torch.equal(attend(cache, batch, q), want)
    with pytest.raises(ValueError, match="bits"):
        cache.bits = 5
        attend(cache, batch, q)


# ------------------------------------------------------------------ workspaces
def work(seed, new=1, length=5000):
    g = gen(seed)
    counts, lengths = [new, new], [length, length // 3]
    starts, table, pages = make_batch(counts, lengths, 64, g)
    cache = full_cache(g, pages, 64, 4, 128, 4)
    return cache, tensors(starts, lengths, table), values(g, 2 * new, 16, 128, dtype=torch.bfloat16)


def test_eager_calls_on_two_streams_at_once():
    """Parts of units that blocks share lie in the workspace between a call's two
    kernels: streams that ran at once over one workspace would mix them."""
    jobs = [work(21), work(22, new=80)]
    want = [attend(*job) for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    outs = [[], []]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(60):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(attend(*jobs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


@pytest.mark.parametrize("shared", [False, True])
def test_eager_calls_from_threads(shared):
    """Four threads, each with a stream of its own or all with one: a call's two
    kernels follow each other in either case."""
    jobs = [work(31 + i, new=1 + 40 * (i % 2)) for i in range(4)]
    want = [attend(*job) for job in jobs]
    torch.cuda.synchronize()
    one, bad = torch.cuda.Stream(), []

    def turn(i):
        try:
            st = one if shared else torch.cuda.Stream()
            with torch.cuda.stream(st):
                outs = [attend(*jobs[i]) for _ in range(40)]
            st.synchronize()
            if not all(torch.equal(o, want[i]) for o in outs):
                bad.append(i)
        except Exception as e:                               # a thread's own would be lost
            bad.append((i, e))

    threads = [threading.Thread(target=turn, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert bad == []


def test_kept_workspaces_are_few():
    """A process that goes round many streams keeps the workspaces of a few."""
    from bit_error_compensated_gb300 import echo
    job = work(41)
    want = attend(*job)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(14)], []
    for _ in range(3):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(attend(*job))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert len(echo._workspaces) <= 4


def test_streams_of_others_have_no_kept_workspace():
    """A raw handle that torch did not make may be another stream's tomorrow."""
    from bit_error_compensated_gb300 import echo
    job = work(42)
    want = attend(*job)
    mine = torch.cuda.Stream()
    other = torch.cuda.ExternalStream(mine.cuda_stream)
    torch.cuda.synchronize()
    before = set(echo._workspaces)
    with torch.cuda.stream(other):
        outs = [attend(*job) for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert set(echo._workspaces) == before
