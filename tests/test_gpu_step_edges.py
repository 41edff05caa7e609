"""Edges of the serving-step operators on the GPU."""
import math
import threading

import pytest
import torch

from _gpu import need_gpu
from test_gpu_step import BF, F32, check, dists, i32, make, on, run_verify

import kimi_delta_attention_chunked_gb300 as kda

pytestmark = pytest.mark.gpu
SLEEP = 20_000_000                                          # cycles, about 10 ms


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (F32, 64)])
@pytest.mark.parametrize("window", [1, 128, 2 ** 31 - 2, 2 ** 31 - 1])
def test_attention_window_of_rows_before_position_zero(dtype, d, window):
    """More new tokens than the sequence holds, under windows up to the largest: the rows
    at and past position 0 see what they see without the others."""
    dev = need_gpu()
    c = make([(-3, 5), (40, 2), (-200, 201), (-150, 460), (-2, 4), (-7, 7), (0, 3)], 8, 2, d, 16, dtype, dev)
    o, lse = check(c, dev, window=window)
    assert bool((o[:3] == 0).all()) and bool((o[3:5] != 0).any())


def test_verify_negative_draft_probability_counts_as_zero():
    """u q < p with q below 0 and p = 0 would let a token stand that the target never gives."""
    dev = need_gpu()
    for dtype in (F32, BF):
        target = torch.zeros(4, 2, 6, dtype=dtype)
        target[:, :, 1], target[:, :, 2] = 0.25, 0.75
        draft = torch.zeros(4, 1, 6, dtype=dtype)
        draft[:, 0, 1] = 1.0
        tokens = torch.tensor([[5], [5], [2], [1]], dtype=torch.int32)
        draft[0, 0, 5], draft[1, 0, 5], draft[2, 0, 2] = -0.5, -math.inf, -0.5
        u = torch.tensor([[0.5, 0.1], [0.5, 0.1], [0.5, 0.1], [0.5, 0.1]])
        got = kda.kda_verify_draft(target.to(dev), draft.to(dev), tokens.to(dev), u.to(dev))
        # rows 0, 1: p = q = 0, the rest max(p - q, 0) is all on token 2; row 2: stands; row 3: 0.5 < 0.25 fails
        assert got[1].tolist() == [1, 1, 2, 1]
        assert got[0].tolist() == [[2, -1], [2, -1], [2, 1], [2, -1]]


def small_verify(dev, n=64):
    return (torch.full((n, 2, 9), 1 / 9, device=dev), None, torch.zeros(n, 1, dtype=torch.int32, device=dev),
            torch.zeros(n, 2, device=dev))


def workspace(args, dtype):
    T, heads, d = args[0].shape
    size = kda.kda_paged_attention_workspace_size(T, heads, args[1].shape[1], d, dtype)
    return torch.empty(size, dtype=torch.uint8, device=args[0].device)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_outputs_of_another_stream_are_not_memory_that_the_current_stream_still_writes(dtype, d):
    """A tensor freed with work of the current stream behind it is not the output of a call
    that another stream runs at once."""
    dev = need_gpu()
    c = make([(300, 2), (90, 30), (5, 1)], 8, 2, d, 32, dtype, dev)
    args = on(c, dev)
    want, want_lse = kda.kda_paged_attention(*args, want_lse=True)
    votes = small_verify(dev)
    want_tokens, want_commit = kda.kda_verify_draft(*votes)
    shapes = [(t.shape, t.dtype) for t in (want, want_lse, want_tokens, want_commit)]
    side = torch.cuda.Stream()
    ws = workspace(args, dtype)
    kda.kda_paged_attention(*args, want_lse=True, workspace=ws, stream=side)         # kernels loaded, pools in use
    kda.kda_verify_draft(*votes, stream=side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    stale = [torch.empty(s, dtype=t, device=dev) for s, t in shapes for _ in range(3)]
    torch.cuda._sleep(SLEEP)
    for t in stale:
        t.fill_(7)                                          # runs after the sleep
    del stale, t
    got = [*kda.kda_paged_attention(*args, want_lse=True, workspace=ws, stream=side),
           *kda.kda_verify_draft(*votes, stream=side)]
    torch.cuda.synchronize()
    for a, b in zip(got, (want, want_lse, want_tokens, want_commit)):
        assert torch.equal(a, b)


def test_outputs_of_another_stream_when_new_memory_is_filled():
    """torch fills new memory where deterministic algorithms are asked for: before the call's
    kernels, not after them."""
    dev = need_gpu()
    c = make([(300, 2), (90, 30)], 8, 2, 128, 32, BF, dev)
    args = on(c, dev)
    want = kda.kda_paged_attention(*args)
    side = torch.cuda.Stream()
    ws = workspace(args, BF)
    torch.cuda.synchronize()
    try:
        torch.use_deterministic_algorithms(True)
        torch.cuda._sleep(SLEEP)
        got = kda.kda_paged_attention(*args, workspace=ws, stream=side)
    finally:
        torch.use_deterministic_algorithms(False)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_memory_of_a_call_on_another_stream_is_kept_until_that_stream_is_done(dtype, d):
    """What a pending call on another stream writes (its workspace, outputs that nobody
    holds any more) is not handed out to the current stream before it has run."""
    dev = need_gpu()
    c = make([(3000, 2), (2000, 30)], 8, 2, d, 32, dtype, dev)
    args = on(c, dev)
    votes = small_verify(dev)
    kda.kda_paged_attention(*args)
    shapes = [(t.shape, t.dtype) for t in (*kda.kda_verify_draft(*votes), args[0], workspace(args, dtype))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    kda.kda_paged_attention(*args, stream=side)
    kda.kda_verify_draft(*votes, stream=side)
    junk = [torch.full(s, 77, dtype=t, device=dev) for s, t in shapes for _ in range(4)]
    torch.cuda.synchronize()
    for t in junk:
        assert bool((t == 77).all())


def test_outputs_read_on_the_current_stream_are_kept_until_it_is_done():
    """An output freed with work of the current stream behind it is not handed out to the
    other stream's next call before that work has run."""
    dev = need_gpu()
    c = make([(300, 2), (90, 30), (5, 1)], 8, 2, 128, 32, BF, dev)
    args = on(c, dev)
    other = [torch.zeros_like(args[0]), *args[1:]]
    want = kda.kda_paged_attention(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = kda.kda_paged_attention(*args, stream=side)
    side.synchronize()
    torch.cuda._sleep(SLEEP)
    read = got.clone()
    del got
    later = [kda.kda_paged_attention(*other, stream=side) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(read, want) and len(later) == 3


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("lens,Hq,Hkv", [
    ([(6000, 32)], 8, 1),                                   # 256 rows, a part in each of 47 CTAs
    ([(3000, 63)], 8, 1),                                   # a full unit and a short one
    ([(1500, 63)], 4, 1),                                   # one unit of 252 rows
    ([(2500, 12), (1, 1), (1300, 20)], 16, 2),
    ([(2300, 9)], 24, 1),                                   # 216 rows, groups that do not fill a tile
])
def test_attention_units_joined_by_all_their_ctas(d, lens, Hq, Hkv):
    """Units of more than 64 rows in many parts."""
    dev = need_gpu()
    c = make(lens, Hq, Hkv, d, 64, BF, dev, seed=d + Hq)
    o, _ = check(c, dev)
    again = kda.kda_paged_attention(*on(c, dev)).double().cpu()
    assert torch.equal(o, again)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("ctas", range(1, 9))
def test_verify_every_cluster_size(dtype, ctas):
    """A row is shared by V / 4096 CTAs, up to eight."""
    dev = need_gpu()
    V = 4096 * ctas + 17 * ctas + 3
    target, draft, tokens, u = dists(2, 2, V, dtype, ctas)
    run_verify(target, draft, tokens, u, [2, 1], dev)
    run_verify(target, None, tokens, u, [1, 2], dev)


def test_calls_at_once_on_two_streams():
    """Attention on the tensor cores and on the CUDA cores, and verification, in two streams at once."""
    dev = need_gpu()
    sets = [make([(900, 2), (90, 30)], 8, 2, 128, 32, BF, dev, seed=1), make([(2000, 1), (40, 9)], 8, 2, 64, 16, BF, dev, seed=2),
            make([(300, 3)], 4, 2, 64, 16, F32, dev, seed=3)]
    args = [on(c, dev) for c in sets]
    votes = small_verify(dev)
    want = [kda.kda_paged_attention(*a) for a in args]
    tokens, _ = kda.kda_verify_draft(*votes)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for i in range(30):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                j = (i + k) % 3
                got.append((kda.kda_paged_attention(*args[j]), want[j]))
                got.append((kda.kda_verify_draft(*votes)[0], tokens))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)
    assert kda.kda_get_last_device_status() == 0


def test_calls_at_once_from_two_threads():
    """The binding gives up the interpreter lock around each call."""
    dev = need_gpu()
    args = on(make([(900, 2), (90, 30)], 8, 2, 128, 32, BF, dev, seed=1), dev)
    votes = small_verify(dev)
    want, tokens = kda.kda_paged_attention(*args), kda.kda_verify_draft(*votes)[0]
    torch.cuda.synchronize()
    bad = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(100):
                o = kda.kda_paged_attention(*args)
                t = kda.kda_verify_draft(*votes)[0]
                with pytest.raises(ValueError):
                    kda.kda_paged_attention(*args[:5], args[5][:1])
            stream.synchronize()
        if not (torch.equal(o, want) and torch.equal(t, tokens)):
            bad.append(threading.get_ident())

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and kda.kda_get_last_device_status() == 0


def test_exception_behind_the_interpreter_lock():
    """A tensor without memory raises, also where its pointer is asked for after the lock was given up."""
    dev = need_gpu()
    args = on(make([(90, 3)], 8, 2, 128, 32, BF, dev), dev)
    want = kda.kda_paged_attention(*args)
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        fake = torch.empty(1 << 28, dtype=torch.uint8, device=dev)
    for _ in range(3):
        with pytest.raises(RuntimeError):
            kda.kda_paged_attention(*args, workspace=fake)
    assert torch.equal(kda.kda_paged_attention(*args), want)


def test_stream_of_another_device_is_refused():
    """A torch stream names its device; the call's tensors have to be there."""
    dev = need_gpu()

    class Elsewhere:
        cuda_stream, device_index = 0, 1

    args = on(make([(20, 3)], 4, 2, 32, 16, F32, dev), dev)
    with pytest.raises(ValueError, match="stream must be on cuda:0, not cuda:1"):
        kda.kda_paged_attention(*args, stream=Elsewhere())
    with pytest.raises(ValueError, match="stream must be on cuda:0"):
        kda.kda_verify_draft(*small_verify(dev), stream=Elsewhere())
    want = kda.kda_paged_attention(*args)
    torch.cuda.synchronize()
    for stream in (torch.cuda.default_stream(), torch.cuda.Stream(), 0, torch.cuda.ExternalStream(torch.cuda.Stream().cuda_stream)):
        got = kda.kda_paged_attention(*args, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_tables_lengths_whose_sums_wrap():
    """Lengths past 2^31 together are outside the contract; the results mean nothing, and
    nothing outside the buffers is written."""
    dev = need_gpu()
    big = 2 ** 31 - 1
    for ctx, new in (([0, 0, 5], [big, big, 7]), ([big, 3, big], [big, big, big]), ([big - 3, 40, 0], [9, big, 40])):
        whole = torch.full((7, 4), 9, dtype=torch.int32, device=dev)
        outs = [torch.full((n + 8,), 9, dtype=t, device=dev) for n, t in
                ((4, torch.int32), (3, torch.int32), (500, torch.int64), (500, torch.int32), (1, torch.int32))]
        kda.kda_build_block_tables(i32(ctx, dev), i32(new, dev), i32([1, 2, 3, 4, 5], dev), whole[2:5], 16, 500,
                                   **dict(zip(("cu_seqlens", "seq_len", "slot_map", "positions", "n_taken"), (o[4:-4] for o in outs))))
        assert bool((whole[:2] == 9).all()) and bool((whole[5:] == 9).all())
        assert all(bool((o[:4] == 9).all()) and bool((o[-4:] == 9).all()) for o in outs)
        slots = outs[2][4:-4]
        assert bool(((slots >= -1) & (slots < 10 * 16)).all())
