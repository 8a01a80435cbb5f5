"""The kernels behind chunk attention and windowed decode at the sizes where they change form:
one query tile per sequence (two key ranges at once), pairs of tiles with several partitions,
groups that do not divide 128, 24 rows in one pass, decode calls with and without a plan kernel;
and calls that share nothing but the device."""

import numpy as np
import pytest
import torch

import paged_kv_cache_422_b200 as nvpa
from tests.window_helpers import ROW_BITS, TILE_BITS, Case, check_answers

pytestmark = pytest.mark.gpu


def _chunk(case, t, num_splits=0, max_q=None, max_ctx=None, **kw):
    return nvpa.chunk_attention(
        t["q"], t["k_cache"], t["v_cache"], t["tables"], t["cu"], t["lens"], max_q or max(case.news),
        max_ctx or max(case.lens), case.scale, window=case.window, num_sinks=case.sinks, k_scales=t["k_scales"],
        v_scales=t["v_scales"], num_splits=num_splits, return_lse=True, **kw)


def _check_chunk(dev, case, num_splits=0, what="", **kw):
    t = case.device(dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = _chunk(case, t, num_splits, err_flag=err, **kw)
    assert err.item() == 0, what
    check_answers(case, out, lse, TILE_BITS, what)
    return t, out, lse


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d,bs,lens,news", [
    # rows = tokens * group between the row kernel's and one tile's; contexts of 1 to 17 key tiles
    (8, 1, 64, 16, [2100, 700, 16, 130, 1], [16, 5, 16, 9, 1]),
    (8, 2, 128, 16, [1300, 257, 0, 33], [32, 32, 0, 31]),
    (2, 2, 128, 256, [900, 128, 129], [128, 100, 127]),
    (7, 1, 64, 64, [640, 300], [18, 11]),
    (10, 2, 64, 32, [515, 77], [25, 25]),
])
def test_one_query_tile_per_sequence(cuda_device, fp8, hq, hkv, d, bs, lens, news):
    case = Case(hq + sum(lens), lens, news, hq, hkv, d, bs, fp8)
    for ns in (0, 1, 2, 5):
        _check_chunk(cuda_device, case, ns, f"splits {ns}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(5, 0), (130, 3), (500, 20), (1000, 200)])
def test_one_query_tile_with_windows(cuda_device, fp8, window, sinks):
    case = Case(window, [1200, 515, 40], [30, 33, 40], 4, 1, 128, 16, fp8, window, sinks)
    for ns in (0, 3):
        _check_chunk(cuda_device, case, ns, f"splits {ns}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d,bs", [(3, 1, 64, 16), (5, 1, 128, 256), (6, 1, 64, 64), (14, 2, 64, 32), (2, 2, 64, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 5)])
def test_pairs_of_tiles_for_any_group(cuda_device, fp8, hq, hkv, d, bs, window, sinks):
    """More tokens than one tile holds, an odd number of tiles, contexts that are no multiple of
    128, so that the tiles of a pair end in different key tiles."""
    case = Case(hq + bs, [430, 333, 300], [150, 333, 31], hq, hkv, d, bs, fp8, window, sinks)
    for ns in (0, 2, 4):
        _check_chunk(cuda_device, case, ns, f"splits {ns}")


@pytest.mark.parametrize("hq,hkv,d,new", [(8, 1, 64, 3), (4, 1, 128, 6), (4, 1, 128, 5), (3, 1, 64, 7), (2, 1, 128, 11)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 4)])
def test_up_to_24_rows_in_one_pass(cuda_device, hq, hkv, d, new, window, sinks):
    case = Case(new, [700, 90, new], [new, new, new], hq, hkv, d, 16, True, window, sinks)
    for ns in (0, 3):
        _check_chunk(cuda_device, case, ns, f"splits {ns}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("batch,hq,hkv", [(1, 4, 4), (128, 2, 1), (129, 2, 1), (200, 4, 2), (30, 16, 8)])
def test_decode_of_few_and_of_many_sequences(cuda_device, fp8, batch, hq, hkv):
    """Lengths of zero and one among others, for calls that fit one round of warps and for calls
    that do not; the bounds that a call gives may be larger than its lengths."""
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in rng.choice([0, 1, 2, 15, 16, 17, 40, 64, 65, 200, 333], size=batch)]
    lens[-1] = 1000
    case = Case(batch, lens, [1] * batch, hq, hkv, 64, 16, fp8, window=300, sinks=2)
    t = case.device(cuda_device)
    for max_ctx in (1000, 1008):
        err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        out, lse = nvpa.paged_decode_attention_window(
            t["q"], t["k_cache"], t["v_cache"], t["tables"], t["lens"], max_ctx, case.scale, window=300, num_sinks=2,
            k_scales=t["k_scales"], v_scales=t["v_scales"], err_flag=err, return_lse=True)
        assert err.item() == 0
        check_answers(case, out, lse, ROW_BITS[fp8], f"bound {max_ctx}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("news", [[3, 2], [40, 7], [200, 129]])
def test_the_same_call_gives_the_same_bits(cuda_device, fp8, news):
    case = Case(3, [1500, 600], news, 4, 2, 128, 16, fp8, window=700, sinks=4)
    t, a, la = _check_chunk(cuda_device, case)
    for _ in range(3):
        b, lb = _chunk(case, t)
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_bad_lengths_and_blocks_on_tiles(cuda_device, fp8):
    dev = cuda_device
    for news, max_q in (([40, 50, 30], 50), ([140, 150, 130], 150)):
        case = Case(11, [200, 300, 260], news, 4, 2, 64, 16, fp8)
        t = case.device(dev)
        good, _ = _chunk(case, t)
        cut = np.cumsum([0] + news)
        for lens in ([200, 301, 260], [200, news[1] - 1, 260], [200, -4, 260]):
            err = torch.zeros(1, dtype=torch.int32, device=dev)
            out = torch.full_like(t["q"], 3.0)
            u = dict(t, lens=torch.tensor(lens, dtype=torch.int32, device=dev))
            _chunk(case, u, err_flag=err, out=out)
            assert err.item() == nvpa.NVPA_FLAG_BAD_LENGTH
            assert torch.equal(out[:cut[1]], good[:cut[1]]) and torch.equal(out[cut[2]:], good[cut[2]:])
            assert (out[cut[1]:cut[2]] == 3.0).all()
        for bad in (case.num_blocks, -1):
            u = dict(t, tables=t["tables"].clone())
            u["tables"][1, 2] = bad
            err = torch.zeros(1, dtype=torch.int32, device=dev)
            out, _ = _chunk(case, u, err_flag=err)
            assert err.item() == nvpa.NVPA_FLAG_BAD_BLOCK_ID
            assert torch.equal(out[:cut[1]], good[:cut[1]]) and torch.equal(out[cut[2]:], good[cut[2]:])
            assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_outputs_that_are_only_16_byte_aligned(cuda_device, fp8):
    case = Case(8, [300, 50], [150, 50], 2, 1, 64, 16, fp8)
    t = case.device(cuda_device)
    flat = torch.zeros(t["q"].numel() + 8, dtype=torch.bfloat16, device=cuda_device)
    out = flat[8:].view(t["q"].shape)
    assert out.data_ptr() % 32 == 16
    _, lse = _chunk(case, t, out=out)
    check_answers(case, out, lse, TILE_BITS, "16-byte aligned")
    assert (flat[:8] == 0).all()


def test_captured_chunk_of_one_tile_with_new_lengths(cuda_device):
    """One captured call, replayed with other context lengths and chunk lengths in its buffers."""
    dev = cuda_device
    cases = [Case(70 + i, lens, news, 4, 1, 128, 16, True, window=400, sinks=4)
             for i, (lens, news) in enumerate((([900, 300], [30, 20]), ([64, 800], [10, 32]), ([31, 0], [31, 0])))]
    ts = [c.device(dev) for c in cases]
    nb, width = max(c.num_blocks for c in cases), max(c.tables.shape[1] for c in cases)
    total = max(c.total for c in cases)
    buf = dict(q=torch.zeros((total, 4, 128), dtype=torch.bfloat16, device=dev), lens=ts[0]["lens"].clone(),
               cu=ts[0]["cu"].clone(), tables=torch.full((2, width), -1, dtype=torch.int32, device=dev))
    for x in "kv":
        buf[x + "_cache"] = torch.zeros((nb, 16, 1, 128), dtype=torch.uint8, device=dev)
        buf[x + "_scales"] = torch.zeros((nb, 1, 16), dtype=torch.uint8, device=dev)

    def load(c, t):
        buf["q"][:c.total] = t["q"]
        buf["lens"].copy_(t["lens"])
        buf["cu"].copy_(t["cu"])
        buf["tables"].fill_(-1)
        buf["tables"][:, :c.tables.shape[1]] = t["tables"]
        for x in "kv":
            buf[x + "_cache"][:c.num_blocks] = t[x + "_cache"].view(torch.uint8)
            buf[x + "_scales"][:c.num_blocks] = t[x + "_scales"]

    ws = torch.empty(nvpa.chunk_attention_workspace_size(2, total, 4, 1, 128, 32, 900, 16, 400, 4), dtype=torch.uint8,
                     device=dev)
    out, lse = torch.zeros_like(buf["q"]), torch.zeros((total, 4), dtype=torch.float32, device=dev)

    def call():
        nvpa.chunk_attention(buf["q"], buf["k_cache"].view(torch.float8_e4m3fn), buf["v_cache"].view(torch.float8_e4m3fn),
                             buf["tables"], buf["cu"], buf["lens"], 32, 900, cases[0].scale, window=400, num_sinks=4,
                             k_scales=buf["k_scales"], v_scales=buf["v_scales"], out=out, lse=lse, workspace=ws,
                             return_lse=True)

    load(cases[0], ts[0])
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in (1, 2, 0, 1):
        load(cases[i], ts[i])
        ws.fill_(0xFF)
        out.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        check_answers(cases[i], out, lse, TILE_BITS, f"replay {i}")
        assert (out[cases[i].total:] == 9).all()


def test_two_streams_at_once_with_their_own_memory(cuda_device):
    """Calls on two side streams that allocate their outputs and workspaces themselves, while the
    current stream reuses memory of its own."""
    dev = cuda_device
    cases = [Case(90, [1500, 900], [20, 30], 4, 1, 64, 16, True), Case(91, [700, 333], [300, 128], 4, 2, 64, 16, False),
             Case(92, [1500, 900], [1, 1], 4, 1, 64, 16, True)]
    ts = [c.device(dev) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for c, t, s in zip(cases, ts, streams):
            got.append((c, _chunk(c, t, stream=s)))
            torch.full((1 << 20,), 7.0, device=dev)
    torch.cuda.synchronize()
    for c, (out, lse) in got:
        check_answers(c, out, lse, TILE_BITS, "streams")


def test_refusals_of_memory_elsewhere(cuda_device):
    dev = cuda_device
    case = Case(1, [40, 20], [30, 5], 4, 2, 64, 16, True)
    t = case.device(dev)
    with pytest.raises(ValueError, match="workspace"):
        _chunk(case, t, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(TypeError, match="workspace"):
        _chunk(case, t, workspace=1 << 20)
    with pytest.raises(ValueError, match="CUDA"):
        _chunk(case, dict(t, cu=t["cu"].cpu()))
    with pytest.raises(TypeError, match="cu_seqlens_q"):
        _chunk(case, dict(t, cu=t["cu"].long()))
    with pytest.raises(ValueError, match="contiguous"):
        _chunk(case, dict(t, q=t["q"].transpose(0, 1).contiguous().transpose(0, 1)))
    with pytest.raises(ValueError, match="batch"):
        _chunk(case, dict(t, cu=t["cu"][:2].contiguous()))
    need = nvpa.chunk_attention_workspace_size(2, 35, 4, 2, 64, 30, 40, 16)
    with pytest.raises(nvpa.NvpaError, match="workspace too small"):
        _chunk(case, t, workspace=torch.empty(need - 256, dtype=torch.uint8, device=dev))
    with pytest.raises(nvpa.NvpaError):
        _chunk(case, t, max_ctx=(1 << 30) + 1)


@pytest.mark.parametrize("fp8", [False, True])
def test_blocks_behind_four_gigabytes(cuda_device, fp8):
    """The same rows in the last blocks of a pool of more than 2^32 bytes and in a small pool:
    equal bits from every call."""
    dev = cuda_device
    hkv, d, bs, used = 8, 128, 256, 5
    row = hkv * d * (1 if fp8 else 2)
    nb = (1 << 32) // (bs * row) + 7
    case = Case(17, [700, 513], [40, 300], 16, hkv, d, bs, fp8, window=600, sinks=4)
    t = case.device(dev)
    assert case.num_blocks >= used
    shift = nb - case.num_blocks
    big = dict(t, tables=torch.where((t["tables"] >= 0) & (t["tables"] < case.num_blocks), t["tables"] + shift, t["tables"]))
    for x in "kv":
        small = t[x + "_cache"]
        pool = torch.empty((nb,) + small.shape[1:], dtype=small.dtype, device=dev)
        pool.view(torch.uint8)[shift:] = small.view(torch.uint8)
        big[x + "_cache"] = pool
        if fp8:
            sc = torch.empty((nb,) + t[x + "_scales"].shape[1:], dtype=torch.uint8, device=dev)
            sc[shift:] = t[x + "_scales"]
            big[x + "_scales"] = sc
    a, la = _chunk(case, t)
    check_answers(case, a, la, TILE_BITS, "small pool")
    b, lb = _chunk(case, big)
    assert torch.equal(a, b) and torch.equal(la, lb)
    # the row kernel: one token per sequence, and two
    for news in ([1, 1], [2, 2]):
        cu = torch.tensor([0, news[0], sum(news)], dtype=torch.int32, device=dev)
        q = t["q"][:sum(news)].contiguous()
        got = []
        for p in (t, big):
            args = (q, p["k_cache"], p["v_cache"], p["tables"])
            kw = dict(window=600, num_sinks=4, k_scales=p["k_scales"], v_scales=p["v_scales"], return_lse=True)
            got.append(nvpa.chunk_attention(*args, cu, t["lens"], news[0], 700, case.scale, **kw) if news[0] > 1 else
                       nvpa.paged_decode_attention_window(*args, t["lens"], 700, case.scale, **kw))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    if fp8:
        # new rows into the last slots, and read back
        g = torch.Generator(device=dev).manual_seed(1)
        k = torch.randn((300, hkv, d), generator=g, device=dev).to(torch.bfloat16)
        slots = torch.arange(nb * bs - 300, nb * bs, dtype=torch.int32, device=dev)
        nvpa.store_kvcache_fp8(k, k, big["k_cache"], big["v_cache"], big["k_scales"], big["v_scales"], slots)
        for x in "kv":
            back = nvpa.gather_kv_fp8(big[x + "_cache"], big[x + "_scales"],
                                      torch.tensor([[nb - 2, nb - 1]], dtype=torch.int32, device=dev),
                                      torch.tensor([0, 512], dtype=torch.int32, device=dev), 512)[-300:]
            # half a step of e4m3, 2^-4 relative, or half the smallest step of the row's scale
            step = torch.exp2(big[x + "_scales"][-2:].double() - 127 - 10).transpose(1, 2).reshape(512, hkv)[-300:, :, None]
            assert ((back.double() - k.double()).abs() <= torch.maximum(2.0 ** -4 * k.double().abs(), step)).all()


def test_sizes_that_do_not_fit_a_c_int_are_refused(cuda_device):
    case = Case(36, [20, 20], [1, 1], 4, 2, 64, 16, True)
    t = case.device(cuda_device)
    pools = (t["q"], t["k_cache"], t["v_cache"], t["tables"])
    sc = dict(k_scales=t["k_scales"], v_scales=t["v_scales"])
    for big in (2 ** 31, 2 ** 32 + 20, 2 ** 40, -2 ** 33):
        for name in ("window", "num_sinks", "num_splits"):
            with pytest.raises(ValueError, match="32 bits"):
                nvpa.paged_decode_attention_window(*pools, t["lens"], 20, 0.125, **sc, **{name: big})
            with pytest.raises(ValueError, match="32 bits"):
                nvpa.chunk_attention(*pools, t["cu"], t["lens"], 1, 20, 0.125, **sc, **{name: big})
        with pytest.raises(ValueError, match="32 bits"):
            nvpa.paged_decode_attention_window(*pools, t["lens"], big, 0.125, **sc)
        with pytest.raises(ValueError, match="32 bits"):
            nvpa.chunk_attention(*pools, t["cu"], t["lens"], big, 20, 0.125, **sc)
