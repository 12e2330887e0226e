"""kv_store with slots that are not different: pieces of 16 bytes, each from one of the slot's
tokens, and no other slot touched.  (Whole rows of one of them are not promised: stores
have no order.)"""
import pytest
import torch

from gpu_util import lib, status_word

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,hkv,d", [(512, 8, 128), (33, 2, 64), (4096, 1, 72)])
def test_pieces_of_the_slots_tokens(cuda, n, hkv, d):
    pkv = lib()
    k = torch.randn((n, hkv, d), device=cuda).to(torch.bfloat16)
    v = torch.randn((n, hkv, d), device=cuda).to(torch.bfloat16)
    kc = torch.full((4, 16, hkv, d), 7.0, dtype=torch.bfloat16, device=cuda)
    vc, st = kc.clone(), pkv.new_status(cuda)
    slots = (torch.arange(n, device=cuda) % 5 * 3).int()
    pkv.kv_store(k, v, kc, vc, slots, status=st)
    assert status_word(st) == 0
    for cache, rows in ((kc, k), (vc, v)):
        flat = cache.view(64, -1, 8)                     # pieces of 16 bytes
        for s in range(64):
            if s % 3 == 0 and s < 15:
                mine = rows[slots == s].view(-1, flat.shape[1], 8)
                assert (mine == flat[s]).all(-1).any(0).all(), s
            else:
                assert (flat[s] == 7).all(), s
