"""bf16 cache, no window: chunk attention and the varlen prefill compute the same attention.  Each is
within the bounds of the same answer, so they differ by at most twice that."""

import numpy as np
import pytest
import torch

import paged_kv_cache_422_b200 as nvpa
from synth.device import i32
from tests.window_helpers import TILE_BITS, Case, check_answers

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,news,hq,hkv,d,bs", [
    ([300, 77, 1], [300, 77, 1], 4, 2, 64, 16),             # whole prompts
    ([700, 257, 130], [200, 257, 129], 8, 2, 128, 256),     # behind cached prefixes
    ([513, 40, 0], [7, 2, 0], 4, 4, 64, 32),                # few rows
    ([900, 300], [70, 20], 16, 2, 128, 64),
])
def test_agrees_with_the_prefill(cuda_device, lens, news, hq, hkv, d, bs):
    case = Case(sum(lens) + d, lens, news, hq, hkv, d, bs, False)
    t = case.device(cuda_device)
    cu_k = i32(np.concatenate([[0], np.cumsum(lens)]), cuda_device)
    ref, ref_lse = nvpa.varlen_prefill_attention(t["q"], t["k_cache"], t["v_cache"], t["tables"], t["cu"], cu_k, max(news),
                                                 max(lens), case.scale, return_lse=True)
    check_answers(case, ref, ref_lse, TILE_BITS, "prefill")
    _, _, ob, mass, lb = case.answers()
    for num_splits in (0, 1, 3):
        out, lse = nvpa.chunk_attention(t["q"], t["k_cache"], t["v_cache"], t["tables"], t["cu"], t["lens"], max(news),
                                        max(lens), case.scale, num_splits=num_splits, return_lse=True)
        off = (out.double() - ref.double()).abs().cpu().numpy()
        assert (off <= 2 * (ob + 2.0 ** -TILE_BITS * mass)).all()
        assert ((lse.double() - ref_lse.double()).abs().cpu().numpy() <= 2 * lb).all()


def test_a_batch_of_a_prompt_chunk_and_single_tokens(cuda_device):
    """A chunk of a prompt beside the next tokens of running sequences, in one call and in two: the
    same answers."""
    dev = cuda_device
    lens, news = [600, 33, 401, 128, 1, 250], [190, 1, 1, 1, 1, 1]
    for fp8 in (False, True):
        case = Case(3, lens, news, 8, 2, 64, 16, fp8, window=0)
        t = case.device(dev)
        sc = dict(k_scales=t["k_scales"], v_scales=t["v_scales"], return_lse=True)
        out, lse = nvpa.chunk_attention(t["q"], t["k_cache"], t["v_cache"], t["tables"], t["cu"], t["lens"], 190, 600,
                                        case.scale, **sc)
        check_answers(case, out, lse, TILE_BITS, "one call")
        a, la = nvpa.chunk_attention(t["q"][:190], t["k_cache"], t["v_cache"], t["tables"][:1], t["cu"][:2], t["lens"][:1],
                                     190, 600, case.scale, **sc)
        b, lb = nvpa.paged_decode_attention_window(t["q"][190:], t["k_cache"], t["v_cache"], t["tables"][1:],
                                                   t["lens"][1:], 600, case.scale, **sc)
        check_answers(case, torch.cat([a, b]), torch.cat([la, lb]), TILE_BITS, "two calls")
