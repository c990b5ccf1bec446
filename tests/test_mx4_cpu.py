"""The 4-bit cache without a GPU: refusals (no kernel is launched by any call here), the layout of a
tile, and the oracle's own answers."""
import ctypes
import subprocess

import pytest
import torch

from jacobi_block_refiner_amd import build, xpress
from tests import mx4_oracle as mx4
from tests.test_serve_abi_cpu import FAKE, ODD2, ODD8, L, cache, says


@pytest.mark.parametrize("code", [2, 3, 15, 18, 32, 1 << 31])
def test_type_codes_of_no_cache_are_refused(code):
    says(L().xpress_cache_trim(cache(dtype=code), None, 4, None, None), b"dtype")
    says(L().xpress_cache_read(cache(dtype=code), 0, None, 4, None, 16, FAKE, FAKE, 1024, None), b"dtype")


@pytest.mark.parametrize("dtype", [xpress.BF16, xpress.F16 + xpress.MX4])
def test_reading_back_checks_its_arguments(dtype):
    c = cache(dtype=dtype)

    def call(c=c, layer=0, seq=None, N=4, first=None, B=16, k=FAKE, v=FAKE, ld=1024):
        return L().xpress_cache_read(c, layer, seq, N, first, B, k, v, ld, None)

    for args, text in ((dict(c=None), b"NULL"), (dict(layer=2), b"layer"), (dict(layer=-1), b"layer"),
                       (dict(seq=ODD2), b"seq"), (dict(N=-1), b"N=-1"), (dict(N=17), b"rows"),
                       (dict(first=ODD2), b"first"), (dict(B=-1), b"B=-1"),
                       (dict(N=16, B=1 << 28), b"2^26"), (dict(k=None), b"k_out"),
                       (dict(k=ODD8), b"k_out"), (dict(v=None), b"v_out"), (dict(v=ODD8), b"v_out"),
                       (dict(ld=1016), b"ld_out"), (dict(ld=1028), b"ld_out")):
        says(call(**args), text)
    assert call(N=0) == xpress.OK and call(B=0) == xpress.OK


@pytest.mark.parametrize("dtype", [xpress.BF16 + xpress.MX4, xpress.F16 + xpress.MX4])
def test_calls_over_four_bits_check_their_arguments(dtype):
    c, size = cache(dtype=dtype), ctypes.c_size_t()
    says(L().xpress_cache_append(c, 0, ODD8, FAKE, 1024, None, 4, 16, None), b"k_new")
    says(L().xpress_cache_append(c, 0, FAKE, FAKE, 1016, None, 4, 16, None), b"ld_new")
    says(L().xpress_cache_extend(c, None, 4, None, 1, FAKE, FAKE, 16, None), b"workspace",
         xpress.ERR_WORKSPACE)
    says(L().xpress_block_attention(c, 0, FAKE, 4096, None, 4, 16, 32, 0.1, 0, FAKE, 4096, None, FAKE, 1,
                                    None), b"workspace", xpress.ERR_WORKSPACE)
    says(L().xpress_block_attention(c, 0, FAKE, 4088, None, 4, 16, 32, 0.1, 0, FAKE, 4096, None, FAKE,
                                    1 << 40, None), b"q_ld")
    assert L().xpress_attention_workspace_size(c, 4, 16, 32, ctypes.byref(size)) == xpress.OK
    assert size.value > 0
    last = 0
    for n in range(16):  # a workspace for more requests serves fewer
        assert L().xpress_attention_workspace_size(c, n, 16, 32, ctypes.byref(size)) == xpress.OK
        assert size.value >= last
        last = size.value


def test_the_binding_refuses_pools_and_tensors():
    pool = torch.zeros(1, 4, 1, 2, 17 * 32, dtype=torch.uint8)
    ok = dict(k=pool, v=pool, table=torch.zeros(2, 3, dtype=torch.int32),
              length=torch.zeros(2, dtype=torch.int32), ref=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(TypeError, match="CUDA"):
        xpress.Cache(**ok)
    with pytest.raises(ValueError, match="17"):
        xpress.Cache(**{**ok, "k": pool[..., :500], "v": pool[..., :500]})
    with pytest.raises(TypeError, match="cannot hold"):
        xpress.Cache(**ok, dtype=torch.float32)
    half = torch.zeros(1, 4, 1, 32, 64, dtype=torch.float16)
    with pytest.raises(TypeError, match="cannot hold"):
        xpress.Cache(**{**ok, "k": half, "v": half}, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="bits"):
        xpress.Cache.empty(1, 4, 1, 16, 64, 2, 3, device="cpu", bits=8)
    with pytest.raises(ValueError, match="4 bits"):
        xpress.Cache.empty(1, 4, 1, 8, 64, 2, 3, device="cpu", bits=4)


LAYOUT = r"""
#include "cache_mx4.hpp"
#include <cstdio>
#include <cmath>
#include <cstring>
#include <initializer_list>
using namespace xpress;
int main() {
  // the bytes of a tile, for a comparison with the definition
  for (int D : {64, 128, 256})
    for (int t = 0; t < 16; ++t) {
      for (int c = 0; c < D; c += 2) printf("%d %d ", mx4_k_code(D, t, c), mx4_v_code(D, t, c));
      for (int g = 0; g < D / 32; ++g) printf("%d %d ", mx4_k_scale(D, t, g), mx4_v_scale(D, t, g));
    }
  if (mx4_tiles_bytes(256, 8) != 16 * 17 * 128 || mx4_tiles_bytes(64, 4) != 17 * 32) return 1;
  // scales: 3.5 to 7 of them hold the largest, inside the limits
  for (bool f16 : {false, true})
    for (int e = -148; e < 128; ++e)
      for (float m : {1.0f, 1.25f, 1.7499999f, 1.75f, 1.9999999f}) {
        const float top = std::ldexp(m, e);
        uint32_t bits;
        std::memcpy(&bits, &top, 4);
        const int s = mx4_scale_byte(bits, f16);
        if (s < mx4_lowest(f16) || s > mx4_highest(f16)) return 2;
        const double times = std::ldexp((double)top, 127 - s);
        if (s > mx4_lowest(f16) && times < 3.5) return 3;
        if (s < mx4_highest(f16) && times >= 7) return 4;
      }
  if (mx4_scale_byte(0, false) != mx4_lowest(false)) return 5;
  if (mx4_scale_byte(0x7f800000u, true) != mx4_highest(true)) return 6;
  // what the limits are for: 6 scales are finite, half the smallest is a value of the type
  if (std::ldexp(6.0, mx4_highest(true) - 127) > 65504 || std::ldexp(0.5, mx4_lowest(true) - 127) < std::ldexp(1.0, -24)) return 7;
  if (std::ldexp(6.0, mx4_highest(false) - 127) > 3.38e38 || std::ldexp(0.5, mx4_lowest(false) - 127) < std::ldexp(1.0, -126)) return 8;
  return 0;
}
"""


def test_the_layout_on_the_host(tmp_path):
    src = tmp_path / "layout.cpp"
    src.write_text(LAYOUT)
    exe = tmp_path / "layout"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover",
                    f"-I{build.CSRC}", str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True)
    assert got.returncode == 0, got.returncode
    want = []
    for D in (64, 128, 256):
        seen = [set(), set()]
        for t in range(16):
            for c in range(0, D, 2):
                want += [mx4.code_byte(D, t, c, v)[0] for v in (False, True)]
            for g in range(D // 32):
                want += [mx4.scale_byte(D, t, g, v) for v in (False, True)]
            for v in (False, True):
                seen[v] |= {mx4.code_byte(D, t, c, v)[0] for c in range(D)}
                seen[v] |= {mx4.scale_byte(D, t, g, v) for g in range(D // 32)}
        assert seen[0] == seen[1] == set(range(17 * D // 2))  # every byte has one meaning
    assert [int(x) for x in got.stdout.split()] == want


def test_the_oracle_on_cases_with_known_answers():
    x = torch.zeros(1, 64, dtype=torch.float64)
    x[0, :11] = torch.tensor([6, 5, 2.5, 3.5, -1.75, 1.25, 0.25, 0.75, -0.2, 7, -0.26])
    x[0, 9] = 6.9  # below 7: the scale stays 1
    x[0, 32:35] = torch.tensor([7.0, 5.0, -0.75])  # a scale of 2
    code, e = mx4.quantise(x, torch.bfloat16)
    assert e.tolist() == [[0, 1]]
    v = mx4.values(code, e)
    assert v[0, :11].tolist() == [6, 4, 2, 4, -2, 1, 0, 1, 0, 6, -0.5]
    assert v[0, 32:35].tolist() == [8, 4, -1] and not v[0, 11:32].any()
    bad = torch.tensor([[float("nan"), float("inf"), -float("inf")] + [1.0] * 29])
    assert mx4.values(*mx4.quantise(bad, torch.float16))[0, :4].tolist() == [0, 49152, -49152, 0]
    y = torch.randn(2, 16, 64, generator=torch.Generator().manual_seed(0))
    for v in (False, True):
        code, e = mx4.quantise(y, torch.bfloat16)
        assert torch.equal(mx4.unpack(mx4.pack(code, e, v), 64, v), mx4.values(code, e))
        far = (mx4.values(code, e) - y.double()).abs().unflatten(-1, (-1, 32))
        assert bool((far <= torch.pow(2.0, e.double())[..., None]).all())  # a scale at most


RUNS = r"""
#include "attend_plan.hpp"
#include <cstdio>
using namespace xpress;
int main() {
  // a wave's walk over the tiles of a pair: every tile once, in order, with its page ids held
  for (int t0 : {0, 1, 5, 63, 64, 1000})
    for (int n = 1; n < 400; ++n) {
      const int t1 = t0 + n;
      int from = t0, seen = t0, rounds = 0;
      for (int t = t0; t < t1;) {
        if (++rounds > n + 1) return 1;  // no way on
        if (few_ids_wanted(t, from, t1)) from = t + 1;
        const int to = few_run_end(t, from, t1);
        if (to <= t || to > t1) return 2;
        for (; t < to; ++t) {
          if (t != seen++) return 3;
          if (t + 1 < t1 && (t + 1 < from || t + 1 - from >= kFewIds)) return 4;
        }
      }
      if (seen != t1) return 5;
      if (rounds > n / (kFewIds - 1) + 2) return 6;
    }
  return 0;
}
"""


def test_a_wave_comes_to_the_end_of_its_tiles(tmp_path):
    src = tmp_path / "runs.cpp"
    src.write_text(RUNS)
    exe = tmp_path / "runs"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover",
                    f"-I{build.CSRC}", f"-I{build.INCLUDE}", str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], timeout=60).returncode == 0
