"""Host-side sizes and checks of attention, the residual update and dropout where there
is nothing, or little, to work on.  No GPU needed: nothing is launched, and the fake
addresses are never dereferenced."""

import ctypes
import subprocess

import pytest
import torch

from adamw_optimizer_step_gb300 import _binding as B
from adamw_optimizer_step_gb300 import build as build_mod
from adamw_optimizer_step_gb300 import layers

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


def attn_args(**kw):
    a = B.AttnArgs()
    o = dict(q=FAKE, k=2 * FAKE, v=3 * FAKE, batch=1, sq=64, sk=64, q_heads=4, k_heads=2, dk=64, dv=64, causal=1,
             dtype=B.GBO_BF16, scale=0.125)
    o.update(kw)
    for k, v in o.items():
        setattr(a, k, v)
    a.q_stride[:], a.k_stride[:], a.v_stride[:] = (64 * 256, 256, 64), (64 * 128, 128, 64), (64 * 128, 128, 64)
    return a


@pytest.mark.parametrize("args", [dict(documents=FAKE), dict(documents=FAKE, n_documents=-1), dict(n_documents=2),
                                  dict(documents=FAKE, n_documents=3, batch=2), dict(documents=FAKE, n_documents=3, sk=65),
                                  dict(documents=FAKE, n_documents=3, k_lengths=FAKE)], ids=str)
def test_attention_sizes_refuse_what_the_calls_refuse(L, args):
    """Documents without a number of them among others: keys are divided among the documents
    to see how a call is cut, so this has to be refused before."""
    a = attn_args(**args)
    for size in (L.gbo_attn_forward_workspace_bytes, L.gbo_attn_backward_workspace_bytes):
        assert size(ctypes.byref(a)) == 0 and b"documents" in L.gbo_last_error()
    assert L.gbo_attn_forward(ctypes.byref(a), 4 * FAKE, a.q_stride, None, None, 0, None, None) == -1


def test_documents_are_two_values_or_more(monkeypatch):
    """One value is the end of no document."""
    class Here:
        """Stands for a CUDA tensor: what the binding asks of one before it packs."""

        def __init__(self, *shape, dtype=torch.bfloat16):
            self.t = torch.zeros(*shape, dtype=dtype)
            self.is_cuda = True

        def __getattr__(self, name):
            return getattr(self.t, name)

        def get_device(self):
            return 0

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    q = Here(1, 5, 2, 8)
    for count in (0, 1):
        with pytest.raises(ValueError, match="documents must be"):
            B.attn_args(q, q, q, documents=Here(count, dtype=torch.int32))
    assert len(B.attn_args(q, q, q, documents=Here(2, dtype=torch.int32))) == ctypes.sizeof(B.AttnArgs)


# how the residual kernels are cut, by a small host program over their header
CUTS = r"""
#include "residual.cuh"

namespace gbo {
int report_error(int code, const char *) { return code; }
int report_ok() { return 0; }
int require_device(int *, int *) { return -1; }
int32_t pdl_allowed() { return 0; }
void count_launches(uint64_t) {}
}  // namespace gbo

int main() {
  using namespace gbo;
  for (int64_t d : {1, 64, 504, 505, 1024, 1031, 4104, 8192, 8199, 16384})
    for (bool back : {false, true})
      for (bool vec : {false, true}) {
        if (vec && d % 8) continue;
        // no rows: no tensors either
        const ResCut c = cut_of(0, d, 152, back, vec, 0);
        if (c.blocks != 1 || c.threads < 32 || c.smem < 0 || c.smem > kSmemMost) return 1;
        if (c.form == kFormRing && (c.stages < 1 || c.stages > kMaxStages)) return 2;
        if (parts_of(c) > most_parts(0, d, 152)) return 3;
        // one row and many, of inputs of any size
        for (int64_t n : {int64_t(1), int64_t(37), int64_t(1) << 40})
          for (int64_t bytes : {16, 1024, 16384, 65536, 163840}) {
            const ResCut r = cut_of(n, d, 152, back, vec, bytes);
            if (r.blocks < 1 || r.blocks > n || r.smem > kSmemMost) return 4;
            if (back && parts_of(r) > most_parts(n, d, 152)) return 5;
            if (r.form == kFormRing && (r.stages < 2 || r.stages > kMaxStages)) return 6;
          }
      }
  return 0;
}
"""


def test_cuts_of_no_rows_and_of_many(tmp_path):
    """A ring's stages are what fits divided by a row's bytes, which are none where there is no row."""
    src, exe = tmp_path / "cuts.cu", tmp_path / "cuts"
    src.write_text(CUTS)
    subprocess.run([build_mod.nvcc(), *build_mod.ARCH, "-std=c++17", "-O1", "--expt-relaxed-constexpr", "-I", build_mod.INCLUDE,
                    "-I", build_mod.CSRC, str(src), "-o", str(exe)], check=True, capture_output=True)
    assert subprocess.run([str(exe)], timeout=60).returncode == 0


# outputs against the arguments that the kernels write them by

def residual_bytes(n, d, gate=B.GBO_GATE_ELEMENT, scale=B.GBO_SCALE_VECTOR, xt=B.GBO_BF16, bt=B.GBO_BF16):
    return bytes(B.ResidualArgs(n=n, d=d, gate_mode=gate, scale_mode=scale, x_dtype=xt, block_dtype=bt, has_block=1))


@pytest.mark.parametrize("modes,what,shape", [
    (dict(scale=B.GBO_SCALE_VECTOR), "dscale", (1,)), (dict(scale=B.GBO_SCALE_ONE), "dscale", (64,)),
    (dict(gate=B.GBO_GATE_ELEMENT), "dgate", (1, 1)), (dict(gate=B.GBO_GATE_ROW), "dgate", (1, 64)),
    (dict(gate=B.GBO_GATE_ROW), "dgate", (2, 1)), (dict(), "dpost_gain", (1,)), (dict(), "dpre_gain", (63,)),
], ids=str)
def test_residual_gradients_have_the_sizes_of_what_they_are_of(monkeypatch, modes, what, shape):
    """A scale of d values has d gradients, not one, whatever the output's own size says."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)  # (where these tensors are)
    out = torch.zeros(shape, dtype=torch.bfloat16 if what == "dgate" else torch.float32)
    with pytest.raises(ValueError, match=what + " must be (1|64|two-dim)"):
        B.gbo_residual_backward(residual_bytes(1, 64, **modes), None, (1, 64), torch.bfloat16, torch.bfloat16, **{what: out})


@pytest.mark.parametrize("shape,xt,bt", [((4, 63), 1, 1), ((5, 64), 1, 1), ((4, 64), 0, 1), ((4, 64), 0, 0)])
def test_residual_outputs_are_of_the_arguments_rows(shape, xt, bt):
    types = [{1: torch.bfloat16, 0: torch.float32}[t] for t in (xt, bt)]
    args = residual_bytes(4, 64)
    with pytest.raises(ValueError, match="args are of"):
        B.gbo_residual_forward(args, None, None, shape, *types)
    with pytest.raises(ValueError, match="args are of"):
        B.gbo_residual_backward(args, None, shape, *types)


@pytest.mark.parametrize("what,shape", [("q", (2, 5, 4, 64)), ("q", (1, 4, 4, 64)), ("k", (1, 7, 1, 64)), ("v", (1, 7, 2, 32)),
                                        ("v", (1, 9, 2, 64))], ids=str)
def test_attention_outputs_are_of_the_arguments_tensors(what, shape):
    """Outputs are checked against the tensors beside the arguments: those have to be the arguments' own."""
    args = bytes(B.AttnArgs(batch=1, sq=5, sk=7, q_heads=4, k_heads=2, dk=64, dv=64))
    shapes = dict(dict(q=(1, 5, 4, 64), k=(1, 7, 2, 64), v=(1, 7, 2, 64)), **{what: shape})
    q, k, v = (torch.zeros(shapes[n], dtype=torch.bfloat16) for n in "qkv")
    dy = torch.zeros(*q.shape[:3], v.shape[3], dtype=torch.bfloat16)
    if what != "k":
        with pytest.raises(ValueError, match="args are of " + what):
            B.gbo_attn_forward(args, q, v, torch.zeros_like(dy))
    with pytest.raises(ValueError, match="args are of " + what):
        B.gbo_attn_backward(args, q, k, v, dy, dy, None, None)


def test_a_stream_without_a_block_is_not_written():
    """The norm alone leaves the stream as it is: a place for the updated one is refused, not ignored."""
    x = torch.zeros(2, 8)
    for t in (x, x.view(1, 2, 8)):
        with pytest.raises(ValueError, match="x_out without"):
            layers.residual_norm(t, x_out=torch.empty_like(t))
