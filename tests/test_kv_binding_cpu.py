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


CALLS = {
    "kv_reserve": lambda a: gdn.kv_reserve(a["lens"], a["add"], a["table"], a["ref"], 16, a["granted"], stream=Stream),
    "kv_append": lambda a: gdn.kv_append(a["k"], a["v"], a["k_pages"], a["v_pages"], a["lens"], a["table"],
                                         count=a["count"], stream=Stream),
    "kv_rollback_tree": lambda a: gdn.kv_rollback_tree(a["node"], a["parent"], a["lens"], a["table"], a["ref"], a["pool"],
                                                       a["lens_out"], count=a["count"], stream=Stream),
    "kv_free": lambda a: gdn.kv_free(a["rows"], a["lens"], a["table"], a["ref"], stream=Stream),
    "kv_fork": lambda a: gdn.kv_fork(a["src"], a["dst"], a["lens"], a["table"], a["ref"], a["pool"], a["granted"],
                                     stream=Stream),
    "kv_compact": lambda a: gdn.kv_compact(a["table"], a["ref"], a["pool"], a["table_out"], a["ref_out"], a["work"],
                                           stream=Stream),
    "kv_copy": lambda a: gdn.kv_copy(a["src"], a["dst"], a["pool"], stream=Stream),
    "attn_verify": lambda a: gdn.attn_verify(a["q"], a["k_pages"], a["v_pages"], a["lens"], a["table"], a["o"],
                                             count=a["count"], parent=a["parent"], lse=a["lse"], workspace=a["work"],
                                             stream=Stream),
}
SHAPES = dict(table=(2, 4), table_out=(2, 4), ref=(8,), ref_out=(8,), pool=(2, 8, 2, 16, 64), k_pages=(8, 2, 16, 64),
              v_pages=(8, 2, 16, 64), q=(2, 3, 4, 64), o=(2, 3, 4, 64), k=(2, 3, 2, 64), v=(2, 3, 2, 64), work=(64,),
              parent=(2, 3), lse=(2, 3, 4))
TYPES = dict(pool=BF, k_pages=BF, v_pages=BF, q=BF, o=BF, k=BF, v=BF, work=torch.uint8, lse=torch.float32)


class Args(dict):
    """Tensors by name, made when a call asks for them: the one called `other` on a second device."""

    def __init__(self, other=None):
        super().__init__()
        self.other = other

    def __missing__(self, name):
        self[name] = fake(*SHAPES.get(name, (2,)), dtype=TYPES.get(name, I32),
                          device="cuda:1" if name == self.other else "cuda:0")
        return self[name]


def tensors_of(name):
    a = Args()
    with pytest.raises(Exception):
        CALLS[name](a)
    return list(a)


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_two_devices(name):
    names = tensors_of(name)
    assert len(names) >= 3
    for other in names:
        with pytest.raises(ValueError, match="one device"):
            CALLS[name](Args(other))
