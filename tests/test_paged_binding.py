"""The binding of the paged-cache operators checks the tensors' lengths before it
calls the library. Stand-in tensors and a stand-in library: no GPU and no call."""
import math

import pytest

from tests.gpu_helpers import built_lib


class Tensor:
    """What the binding asks of a device tensor."""
    is_cuda = True

    def __init__(self, dtype, *shape, row_stride=None):
        self.dtype, self.shape, self.row_stride = "torch." + dtype, shape, row_stride

    def is_contiguous(self):
        return self.row_stride is None

    def numel(self):
        return math.prod(self.shape)

    def dim(self):
        return len(self.shape)

    def stride(self, i):
        return (self.row_stride, 1)[i]

    def data_ptr(self):
        return 1 << 20


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def B(monkeypatch):
    built_lib()
    from q8_quantized_llama_gb300 import binding
    stub = Library()
    monkeypatch.setattr(binding, "lib", lambda: stub)
    monkeypatch.setattr(binding, "stub", stub, raising=False)
    return binding


ROWS, N_SEQ, WIDTH, HEADS, KV, DIM, PAGES = 5, 6, 7, 6, 2, 64, 40


def _pages(B):
    t = Tensor("float16", 3, PAGES, KV, 16, DIM)
    return B.make_pages(t, t)


def _rope(B, t):
    B.llama_q8_rope_append(_pages(B), 0, t["qkv"], 700, ROWS, t["pos"], t["seq"], HEADS,
                           B.make_rope(Tensor("float64", 32)), t["table"], N_SEQ, WIDTH, t["q_out"], t["err"])


def _attention(B, t):
    B.llama_q8_attention_paged(_pages(B), 0, t["q"], ROWS, t["pos"], t["seq"], HEADS, 0.0, 0, t["table"], N_SEQ, WIDTH,
                               t["out"], t["lse"], t["ws"], 1000, t["err"])


def _fork(B, t):
    B.llama_q8_pages_fork(_pages(B), N_SEQ, t["len_in"], t["table_in"], WIDTH, t["refs_in"], ROWS, t["parent"], 1,
                          t["len_out"], t["table_out"], t["refs_out"], t["ws"], 1000, t["err"])


def _compact(B, t):
    B.llama_q8_pages_compact(_pages(B), N_SEQ, t["table_in"], WIDTH, t["refs_in"], t["table_out"], t["refs_out"],
                             t["n_used"], t["ws"], 1000, t["err"])


def _beam(B, t):
    B.llama_q8_beam_select(t["logits"], 120, 3, 4, 100, t["scores"], 5, t["out_scores"], t["parent"], t["token"],
                           t["ws"], 1000)


I, F = "int32", "float32"
CALLS = [
    (_rope, dict(qkv=(F, 4 * 700 + 10 * DIM), pos=(I, ROWS), seq=(I, ROWS), table=(I, N_SEQ * WIDTH),
                 q_out=(F, ROWS * HEADS * DIM), err=(I, 1))),
    (_attention, dict(q=(F, ROWS * HEADS * DIM), pos=(I, ROWS), seq=(I, ROWS), table=(I, N_SEQ * WIDTH),
                      out=(F, ROWS * HEADS * DIM), lse=(F, ROWS * HEADS), ws=("uint8", 1000), err=(I, 1))),
    (_fork, dict(len_in=(I, N_SEQ), table_in=(I, N_SEQ * WIDTH), refs_in=(I, PAGES), parent=(I, ROWS),
                 len_out=(I, ROWS), table_out=(I, ROWS * WIDTH), refs_out=(I, PAGES), ws=("uint8", 1000), err=(I, 1))),
    (_compact, dict(table_in=(I, N_SEQ * WIDTH), refs_in=(I, PAGES), table_out=(I, N_SEQ * WIDTH), refs_out=(I, PAGES),
                    n_used=(I, 1), ws=("uint8", 1000), err=(I, 1))),
    (_beam, dict(logits=(F, 11 * 120 + 100), scores=(F, 12), out_scores=(F, 15), parent=(I, 15), token=(I, 15),
                 ws=("uint8", 1000)))]


@pytest.mark.parametrize("call,sizes", CALLS)
def test_tensors_of_the_least_length_pass(B, call, sizes):
    call(B, {k: Tensor(*v) for k, v in sizes.items()})
    assert len(B.stub.calls) == 1


@pytest.mark.parametrize("call,sizes,name", [(c, s, n) for c, s in CALLS for n in s if n not in ("ws", "err")])
def test_tensors_that_are_too_short_are_refused(B, call, sizes, name):
    t = {k: Tensor(*v) for k, v in sizes.items()}
    t[name] = Tensor(sizes[name][0], sizes[name][1] - 1)
    with pytest.raises(ValueError, match="values"):
        call(B, t)
    assert not B.stub.calls


@pytest.mark.parametrize("call,sizes,name,rows,width,stride", [(*CALLS[0], "qkv", ROWS, 10 * DIM, 700),
                                                               (*CALLS[4], "logits", 12, 100, 120)])
def test_strided_rows_have_enough_rows_and_values(B, call, sizes, name, rows, width, stride):
    t = {k: Tensor(*v) for k, v in sizes.items()}
    for less in ((1, 0), (0, 1)):
        t[name] = Tensor(F, rows - less[0], width - less[1], row_stride=stride)
        with pytest.raises(ValueError, match="rows"):
            call(B, t)
    assert not B.stub.calls
    t[name] = Tensor(F, rows, width, row_stride=stride)
    call(B, t)
    assert len(B.stub.calls) == 1
