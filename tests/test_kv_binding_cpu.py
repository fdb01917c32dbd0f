"""What the compiled binding of the cache and attention calls turns down by
itself, on tensors that have a device, a type and a shape but no memory (a call
that got through would be refused by the library for its null pointers)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from speculative_verify_gdn_amd import gdn

I32, BF = torch.int32, torch.bfloat16


class Stream:
    cuda_stream = 0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    try:
        gdn.load()
    except FileNotFoundError as e:
        pytest.skip(str(e))


def fake(*shape, dtype=I32, device="cuda:0"):
    with FakeTensorMode():
        return torch.empty(*shape, dtype=dtype, device=device)


def args():
    plane = fake(8, 2, 16, 64, dtype=BF)
    return dict(i=fake(2), table=fake(2, 4), ref=fake(8), pool=fake(2, 8, 2, 16, 64, dtype=BF), k_pages=plane, v_pages=plane,
                q=fake(2, 3, 4, 64, dtype=BF), o=fake(2, 3, 4, 64, dtype=BF), k=fake(2, 3, 2, 64, dtype=BF),
                work=fake(64, dtype=torch.uint8))


@pytest.mark.parametrize("page", [2 ** 32 + 16, 2 ** 31, -2 ** 32 + 16, 2 ** 70])
def test_page_past_32_bits(page):
    a = args()
    with pytest.raises(ValueError, match="page"):
        gdn.kv_reserve(a["i"], a["i"], a["table"], a["ref"], page, a["i"], stream=Stream)


@pytest.mark.parametrize("N", [2 ** 32 + 4, 2 ** 31, -2 ** 40])
def test_window_length_past_32_bits(N):
    a = args()
    with pytest.raises(ValueError, match="N"):
        gdn.kv_rollback_tree(a["i"], None, a["i"], a["table"], a["ref"], a["pool"], a["i"], N=N, stream=Stream)


@pytest.mark.parametrize("prefix", [2 ** 32 + 16, 2 ** 31, 2 ** 80])
def test_prefix_past_32_bits(prefix):
    a = args()
    with pytest.raises(ValueError, match="prefix_len"):
        gdn.attn_verify(a["q"], a["k_pages"], a["v_pages"], a["i"], a["table"], a["o"], prefix_len=prefix,
                        workspace=a["work"], stream=Stream)


def test_not_numbers():
    a = args()
    with pytest.raises(TypeError):
        gdn.kv_reserve(a["i"], a["i"], a["table"], a["ref"], "16", a["i"], stream=Stream)
    with pytest.raises(TypeError):
        gdn.kv_reserve(a["i"], a["i"], a["table"], a["ref"], 16.0, a["i"], stream=Stream)
