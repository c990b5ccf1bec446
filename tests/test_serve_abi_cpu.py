"""The target's side of a draft step without a GPU: argument errors are found on the host (no kernel
is launched by any call here), and the cache's index arithmetic is right at its limits."""
import ctypes
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

from jacobi_block_refiner_amd import build, xpress
from tests.serve_oracle import CacheOracle, attention, verify

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
ODD2 = ctypes.c_void_p((1 << 20) + 2)
ODD8 = ctypes.c_void_p((1 << 20) + 8)
GOOD = dict(n_layers=2, n_pages=64, page=64, Hkv=8, D=128, dtype=xpress.BF16, rows=16, table_ld=32,
            k=FAKE, v=FAKE, table=FAKE, len=FAKE, ref=FAKE)


def cache(**change):
    return ctypes.byref(xpress._Cache(**{**GOOD, **change}))


def L():
    return xpress.lib()


def says(status, text, want=xpress.ERR_ARG):
    assert status == want
    assert text in L().xpress_last_error(), L().xpress_last_error()


BAD_CACHES = [(dict(n_layers=0), b"n_layers"), (dict(n_layers=65537), b"n_layers"), (dict(n_pages=0), b"n_pages"),
              (dict(n_pages=(1 << 24) + 1), b"n_pages"), (dict(page=8), b"page"),
              (dict(page=48), b"page"), (dict(Hkv=0), b"Hkv"), (dict(Hkv=257), b"Hkv"),
              (dict(D=96), b"D="), (dict(dtype=xpress.F32), b"dtype"), (dict(rows=0), b"rows"),
              (dict(table_ld=0), b"table_ld"), (dict(table_ld=(1 << 20) + 1), b"table_ld")]


@pytest.mark.parametrize("change,text", BAD_CACHES)
def test_bad_caches_are_refused_by_every_call(change, text):
    c, size = cache(**change), ctypes.c_size_t()
    says(L().xpress_cache_workspace_size(c, 4, ctypes.byref(size)), text)
    says(L().xpress_attention_workspace_size(c, 4, 16, 32, ctypes.byref(size)), text)
    says(L().xpress_cache_fork(c, FAKE, FAKE, 2, None), text)
    says(L().xpress_cache_extend(c, None, 4, None, 16, FAKE, FAKE, 1 << 30, None), text)
    says(L().xpress_cache_append(c, 0, FAKE, FAKE, 1024, None, 4, 16, None), text)
    says(L().xpress_cache_trim(c, None, 4, None, None), text)
    says(L().xpress_cache_compact(c, FAKE, FAKE, 1 << 30, None), text)
    says(L().xpress_block_attention(c, 0, FAKE, 4096, None, 4, 16, 32, 0.1, 0, FAKE, 4096, None,
                                    FAKE, 1 << 30, None), text)


def test_null_and_misaligned_cache_pointers():
    for name in ("k", "v"):
        for p, text in ((None, b"NULL"), (ODD8, b"16-byte")):
            says(L().xpress_cache_append(cache(**{name: p}), 0, FAKE, FAKE, 1024, None, 4, 16,
                                         None), text)
    for name in ("table", "len", "ref"):
        for p, text in ((None, b"NULL"), (ODD2, b"4-byte")):
            says(L().xpress_cache_trim(cache(**{name: p}), None, 4, None, None), text)
    says(L().xpress_cache_trim(None, None, 4, None, None), b"NULL")


def test_cache_calls_check_their_arguments():
    c = cache()
    says(L().xpress_cache_fork(c, None, FAKE, 2, None), b"src")
    says(L().xpress_cache_fork(c, FAKE, ODD2, 2, None), b"dst")
    says(L().xpress_cache_fork(c, FAKE, FAKE, 17, None), b"n=17")
    says(L().xpress_cache_fork(c, FAKE, FAKE, -1, None), b"n=-1")
    says(L().xpress_cache_extend(c, None, 17, None, 1, FAKE, FAKE, 1 << 30, None), b"rows")
    says(L().xpress_cache_extend(c, None, -1, None, 1, FAKE, FAKE, 1 << 30, None), b"N=-1")
    says(L().xpress_cache_extend(c, None, 4, None, -1, FAKE, FAKE, 1 << 30, None), b"add_all")
    says(L().xpress_cache_extend(c, None, 4, None, 1, None, FAKE, 1 << 30, None), b"lacking")
    says(L().xpress_cache_extend(c, None, 4, None, 1, FAKE, None, 1 << 30, None), b"ws")
    says(L().xpress_cache_extend(c, None, 4, None, 1, FAKE, FAKE, 16, None), b"workspace",
         xpress.ERR_WORKSPACE)
    says(L().xpress_cache_append(c, 2, FAKE, FAKE, 1024, None, 4, 16, None), b"layer")
    says(L().xpress_cache_append(c, -1, FAKE, FAKE, 1024, None, 4, 16, None), b"layer")
    says(L().xpress_cache_append(c, 0, FAKE, FAKE, 1016, None, 4, 16, None), b"ld_new")
    says(L().xpress_cache_append(c, 0, FAKE, FAKE, 1028, None, 4, 16, None), b"ld_new")
    says(L().xpress_cache_append(c, 0, ODD8, FAKE, 1024, None, 4, 16, None), b"k_new")
    says(L().xpress_cache_append(c, 0, FAKE, FAKE, 1024, None, 16, 1 << 28, None), b"2^26")
    says(L().xpress_cache_trim(c, ODD2, 4, None, None), b"seq")
    says(L().xpress_cache_compact(c, None, FAKE, 1 << 30, None), b"live")
    says(L().xpress_cache_compact(c, FAKE, FAKE, 64, None), b"workspace", xpress.ERR_WORKSPACE)


def test_attention_checks_its_arguments():
    def call(c=None, layer=0, q=FAKE, q_ld=4096, seq=None, N=4, B=16, Hq=32, scale=0.1, shared=0,
             out=FAKE, out_ld=4096, lse=None, ws=FAKE, ws_bytes=1 << 40):
        return L().xpress_block_attention(c or cache(), layer, q, q_ld, seq, N, B, Hq, scale, shared,
                                          out, out_ld, lse, ws, ws_bytes, None)

    for args, text in ((dict(layer=2), b"layer"), (dict(N=-1), b"N=-1"), (dict(N=17), b"rows"),
                       (dict(B=0), b"B=0"), (dict(Hq=0), b"Hq"), (dict(Hq=12), b"Hq"),
                       (dict(B=1 << 24), b"2^26"), (dict(q_ld=4088), b"q_ld"),
                       (dict(q_ld=4100), b"q_ld"), (dict(out_ld=4100), b"out_ld"),
                       (dict(scale=0.0), b"scale"), (dict(scale=-1.0), b"scale"),
                       (dict(scale=float("nan")), b"scale"), (dict(scale=1e7), b"scale"),
                       (dict(shared=-1), b"shared"), (dict(shared=32 * 64 + 1), b"shared"),
                       (dict(q=None), b"q is NULL"), (dict(q=ODD8), b"16-byte"),
                       (dict(out=ODD8), b"16-byte"), (dict(lse=ODD2), b"lse"),
                       (dict(seq=ODD2), b"seq"), (dict(ws=None), b"ws")):
        says(call(**args), text)
    says(call(ws_bytes=1), b"workspace", xpress.ERR_WORKSPACE)
    assert call(N=0) == xpress.OK


def test_attention_workspace_for_n_max_fits_every_smaller_n():
    size = ctypes.c_size_t()

    def need(n, B, Hq, **change):
        assert L().xpress_attention_workspace_size(cache(rows=4096, **change), n, B, Hq,
                                                   ctypes.byref(size)) == xpress.OK
        return size.value

    for change in ({}, dict(table_ld=4096), dict(page=16, table_ld=3), dict(Hkv=1), dict(D=256)):
        for B, G in ((1, 1), (16, 5), (7, 3), (1, 16), (256, 1)):
            Hq = G * change.get("Hkv", 8)
            most = 0
            for n in range(0, 400, 3):
                most = max(most, need(n, B, Hq, **change))
                assert need(n, B, Hq, **change) >= most, (change, B, G, n)


def test_verify_checks_its_arguments():
    def call(logits=FAKE, dtype=xpress.BF16, ld=1000, blk=FAKE, dl=None, q=None, qt=xpress.F32,
             q_ld=1000, temperature=FAKE, u=FAKE, N=4, B=16, V=1000, out=FAKE, accepted=FAKE,
             drop=None, ws=FAKE, ws_bytes=1 << 40):
        return L().xpress_verify_draft(logits, dtype, ld, blk, dl, q, qt, q_ld, temperature, u, N, B,
                                       V, out, accepted, drop, ws, ws_bytes, None)

    odd1 = ctypes.c_void_p((1 << 20) + 1)
    for args, text in ((dict(logits=None), b"logits"), (dict(logits=odd1), b"aligned"),
                       (dict(dtype=3), b"type"), (dict(dtype=xpress.F32, logits=ODD2), b"aligned"),
                       (dict(ld=999), b"stride"), (dict(q=FAKE, qt=9), b"q: unknown"),
                       (dict(q=FAKE, q_ld=10), b"q: row stride"), (dict(q=ODD2), b"q is not"),
                       (dict(blk=None), b"blk"), (dict(out=None), b"out"), (dict(blk=ODD2), b"blk"),
                       (dict(accepted=None), b"accepted"), (dict(drop=ODD2), b"drop"),
                       (dict(dl=ODD2), b"draft_len"), (dict(u=None), b"u is NULL"),
                       (dict(N=-1), b"N=-1"), (dict(B=0), b"B=0"), (dict(B=65), b"B=65"),
                       (dict(V=0), b"V=0"), (dict(V=1 << 31), b"V="), (dict(ws=None), b"ws")):
        says(call(**args), text)
    says(call(ws_bytes=1), b"workspace", xpress.ERR_WORKSPACE)
    assert call(N=0) == xpress.OK


def test_verify_workspace_grows_with_rows():
    size, last = ctypes.c_size_t(), 0
    for n in range(1, 300):
        assert L().xpress_verify_workspace_size(n, 16, 151936, ctypes.byref(size)) == xpress.OK
        assert size.value >= last
        last = size.value
    says(L().xpress_verify_workspace_size(1, 16, 0, ctypes.byref(size)), b"V=0")
    says(L().xpress_verify_workspace_size(1, 16, 10, None), b"bytes")


def test_binding_refuses_host_tensors_and_shapes():
    shape = (1, 4, 1, 16, 64)
    k = torch.zeros(shape, dtype=torch.bfloat16)
    ok = dict(k=k, v=k, table=torch.zeros(2, 3, dtype=torch.int32),
              length=torch.zeros(2, dtype=torch.int32), ref=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(TypeError, match="CUDA"):
        xpress.Cache(**ok)
    for change, error in ((dict(v=k[:, :2]), ValueError), (dict(length=torch.zeros(3)), ValueError),
                          (dict(ref=torch.zeros(5)), ValueError),
                          (dict(k=k.float(), v=k.float()), TypeError)):
        with pytest.raises(error):
            xpress.Cache(**{**ok, **change})
    blk = torch.zeros(2, 3, dtype=torch.int64)
    with pytest.raises(TypeError):
        xpress.verify_draft(torch.zeros(6, 10), blk, out=blk, accepted=blk, ws=blk)
    with pytest.raises(TypeError):
        xpress.verify_draft(torch.zeros(6, 10, dtype=torch.int8), blk, out=blk, accepted=blk, ws=blk)


INDEX = r"""
#include "cache_index.hpp"
#include <cstdio>
#include <climits>
#include <initializer_list>
using namespace xpress;
int main() {
  // pages of a token count, up to the largest table
  for (int s = 4; s <= 8; ++s)
    for (long long n : {0LL, 1LL, (1LL << s) - 1, 1LL << s, (1LL << s) + 1, (1LL << 30) + 1})
      if (pages_of(n, s) != (int)((n + (1LL << s) - 1) / (1LL << s))) return 1;
  // lengths stay inside the table, whatever the buffer holds
  for (int len : {INT_MIN, -1, 0, 5, 1 << 20, INT_MAX})
    for (int ld : {1, 7, 1 << 20}) {
      const int got = clamp_len(len, ld, 4);
      if (got < 0 || got > (long long)ld * 16) return 2;
      if (len >= 0 && len <= (long long)ld * 16 && got != len) return 3;
      if (pages_of(got, 4) > ld) return 4;
    }
  // the longest table of the largest pages still fits an int
  if (clamp_len(INT_MAX, 1 << 20, 8) < 0 || pages_of(clamp_len(INT_MAX, 1 << 20, 8), 8) > 1 << 20) return 5;
  // ids stay inside the pool
  for (int id : {INT_MIN, -1, 0, 6, 7, INT_MAX}) {
    const int got = clamp_page(id, 7);
    if (got < 0 || got >= 7 || page_ok(id, 7) != (got == id)) return 6;
  }
  // offsets past 32 bits
  if (line_offset((1 << 24) - 1, 255, 255, 256, 8, 256) !=
      ((((1LL << 24) - 1) * 256 + 255) * 256 + 255) * 256) return 7;
  // what a query sees
  if (in_sight(0, 16, 15) != 0 || in_sight(1, 16, 15) != 1 || in_sight(1, 16, 14) != 0 ||
      in_sight(20, 16, 0) != 5 || in_sight(INT_MAX, 1, 0) != INT_MAX) return 8;
  return 0;
}
"""


def test_index_arithmetic_on_the_host(tmp_path):
    src = tmp_path / "index.cpp"
    src.write_text(INDEX)
    exe = tmp_path / "index"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover",
                    f"-I{build.CSRC}", str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


PLAN = r"""
#include "attend_plan.hpp"
#include <cstdio>
#include <initializer_list>
using namespace xpress;
int main() {
  xpress_cache c = {};
  for (int D : {64, 128, 256}) for (int page : {16, 256}) for (int Hkv : {1, 2, 8, 32})
  for (int64_t cap : {16LL, 100LL, 700LL, 5000LL, 20000LL, 70000LL, 1LL << 20}) {
    c.D = D, c.page = page, c.Hkv = Hkv, c.table_ld = (cap + page - 1) / page;
    cap = (int64_t)c.table_ld * page;
    for (int G : {1, 5, 16}) for (int B : {1, 3, 16, 64}) {
      int64_t last = 0;
      for (int N : {1, 2, 5, 31, 64, 257, 1000, 4096}) {
        const int64_t most = most_row_slots(c, N, B, Hkv * G);
        if (most < last) return 1;  // a workspace for more requests serves fewer
        last = most;
        for (int64_t sh : {0LL, 64LL, 640LL, 4096LL, 19968LL, 65536LL, 1LL << 20}) {
          if (sh > cap) continue;
          const AttendPlan p = plan_of(c, N, B, Hkv * G, (int)(sh / kTile * kTile));
          if ((int64_t)p.slots() * N > most) {
            printf("D %d page %d Hkv %d cap %lld G %d B %d N %d shared %lld: %d slots, %lld rows\n", D,
                   page, Hkv, (long long)cap, G, B, N, (long long)sh, p.slots(), (long long)most);
            return 2;
          }
          // every key of the shared part in one split, every row in one tile, ids that fit
          if (sh >= kTile && ((int64_t)p.s_sh * p.chunk_sh < sh / kTile * kTile || p.chunk_sh % 32 ||
                              p.chunk_sh / page + 2 > kIds)) return 3;
          if (sh >= kTile && (int64_t)p.tiles_sh * (p.wide ? kWide : kNarrow) * 32 < (int64_t)N * B * G)
            return 4;
          if ((int64_t)p.tiles_own * kNarrow * 32 < (int64_t)B * G || p.s_own < 1) return 5;
          const int64_t own = std::max(cap - sh / kTile * kTile, std::min<int64_t>(cap, sh / kTile * kTile + B));
          const int64_t chunk = ((own + p.s_own - 1) / p.s_own + 63) / 64 * 64;
          if (chunk / page + 2 > kIds) return 6;
        }
      }
    }
  }
  return 0;
}
"""


def test_the_workspace_covers_every_split(tmp_path):
    """The partial results of every plan fit in the workspace that is asked for, also when it was
    asked for with more requests, and an item's page ids fit where the kernel keeps them."""
    src = tmp_path / "plan.cpp"
    src.write_text(PLAN)
    exe = tmp_path / "plan"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover",
                    f"-I{build.CSRC}", f"-I{build.INCLUDE}", str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True)
    assert got.returncode == 0, (got.returncode, got.stdout)


def test_oracles_on_cases_with_known_answers():
    """The oracles themselves: one token's attention is its value; a causal block; a fork that is
    extended; verification by hand."""
    k = torch.zeros(2, 1, 16, 64)
    v = torch.arange(16.0).view(1, 1, 16, 1).expand(2, 1, 16, 64).contiguous()
    q = torch.ones(2, 64)
    out, lse, mass, _ = attention(k, v, np.array([[1]]), [3], 16, q, [0], 2, 1, 0.125)
    assert torch.allclose(out[:, 0, 0], torch.tensor([0.5, 1.0], dtype=torch.float64))
    assert np.allclose(lse[:, 0].numpy(), np.log([2, 3])) and torch.equal(out, mass)
    o = CacheOracle(1, 4, 1, 16, 64, 2, 3, torch.bfloat16)
    assert o.extend([0], [17]) == 0 and o.ref.tolist() == [1, 1, 0, 0]
    o.fork([0], [1])
    assert o.ref.tolist() == [2, 2, 0, 0]
    assert o.extend([1], [1]) == 0 and o.ref.tolist() == [2, 1, 1, 0]
    assert torch.equal(o.k[0, 2], o.k[0, 1])
    o.trim([0], None)
    assert o.ref.tolist() == [1, 0, 1, 0] and o.compact() == 2
    assert o.table.tolist() == [[-1, -1, -1], [0, 1, -1]]
    x = np.log(np.array([[0.5, 0.25, 0.25], [0.1, 0.1, 0.8]]))
    blk = np.array([[0, 1]])
    t = np.ones(1)
    assert verify(x, blk, None, None, t, np.array([[0.2, 0.5]]))[0].tolist() == [[1, 2]]
    assert verify(x, blk, None, None, t, np.array([[0.3, 0.5]]))[0].tolist() == [[0, -1]]
    assert verify(x, blk, None, None, t, np.array([[0.3, 0.7]]))[0].tolist() == [[2, -1]]
    q1 = np.array([[0.2, 0.8, 0.0]])
    assert verify(x, blk, None, q1, t, np.array([[0.3, 0.5]]))[0].tolist() == [[1, 2]]
    assert verify(x, blk, None, q1, t, np.array([[0.4, 0.6]]))[0].tolist() == [[2, -1]]


COUNTS = r"""
#include "cache_index.hpp"
#include <cstdio>
#include <vector>
using namespace xpress;
int main() {
  uint32_t seed = 1;
  for (int turn = 0; turn < 20000; ++turn) {
    auto next = [&] { return (seed = seed * 1664525u + 1013904223u) >> 16; };
    const int n = 1 + next() % 40;
    std::vector<int> ref(n);
    for (int& r : ref) r = (int)(next() % 6) - 2;  // -2 .. 3 holders
    int live = 0, out = 0, in = 0;
    for (int r : ref) live += holders(r) > 0;
    for (int p = 0; p < n; ++p) {
      if (holders(ref[p]) < 0 || (ref[p] >= 0 && holders(ref[p]) != ref[p])) return 1;
      if (moves_out(ref[p], p, live) && takes_in(ref[p], p, live)) return 2;
      // in the front a page is live or takes one in; past it a page moves out or is free
      if ((holders(ref[p]) > 0) == (p < live ? takes_in(ref[p], p, live) : !moves_out(ref[p], p, live)))
        return 3;
      out += moves_out(ref[p], p, live);
      in += takes_in(ref[p], p, live);
    }
    if (out != in) {
      printf("turn %d: %d pages move, %d take them in\n", turn, out, in);
      return 4;
    }
  }
  return 0;
}
"""


def test_a_compaction_has_a_place_for_every_page_it_moves(tmp_path):
    """Whatever the counts, below 0 too (after a row twice in a list): no move without a target."""
    src = tmp_path / "counts.cpp"
    src.write_text(COUNTS)
    exe = tmp_path / "counts"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover",
                    f"-I{build.CSRC}", str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True)
    assert got.returncode == 0, (got.returncode, got.stdout)


def test_conditional_cache_calls_check_their_arguments():
    c = cache()
    says(L().xpress_cache_append_if(c, ODD2, 0, FAKE, FAKE, 1024, None, 4, 16, None), b"lacking")
    says(L().xpress_cache_append_if(c, FAKE, 2, FAKE, FAKE, 1024, None, 4, 16, None), b"layer")
    says(L().xpress_cache_append_if(c, FAKE, 0, ODD8, FAKE, 1024, None, 4, 16, None), b"k_new")
    says(L().xpress_cache_trim_if(c, ODD2, None, 4, None, None), b"lacking")
    says(L().xpress_cache_trim_if(c, FAKE, ODD2, 4, None, None), b"seq")
    says(L().xpress_cache_trim_if(c, FAKE, None, 17, None, None), b"rows")
    assert L().xpress_cache_append_if(c, None, 0, FAKE, FAKE, 1024, None, 0, 16, None) == xpress.OK
    assert L().xpress_cache_trim_if(c, FAKE, None, 0, None, None) == xpress.OK


MISSING = r"""
#include "cache_index.hpp"
#include <initializer_list>
using namespace xpress;
int main() {
  for (int64_t found : {0LL, 1LL, 1LL << 24})
    for (int64_t more : {0LL, 1LL, (1LL << 31) - 1, 1LL << 31, 1LL << 32, 3LL << 32, 1LL << 40})
      if (pages_missing(found + more, found) != (more < INT32_MAX ? (int)more : INT32_MAX)) return 1;
  return pages_missing(3, 5) == 0 ? 0 : 2;
}
"""


def test_missing_pages_past_32_bits(tmp_path):
    """2^20 rows may ask for 2^20 pages each: the number that is missing does not wrap round to 0."""
    src = tmp_path / "missing.cpp"
    src.write_text(MISSING)
    exe = tmp_path / "missing"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover",
                    f"-I{build.CSRC}", str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_the_stream_of_a_torch_without_the_raw_handle():
    """The binding loads and takes the public call's stream where torch lacks the function that gives
    the handle alone."""
    code = """
import torch
from types import SimpleNamespace
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
torch.cuda.current_stream = lambda: SimpleNamespace(cuda_stream=123)
from jacobi_block_refiner_amd import xpress
assert xpress._stream() == 123
"""
    got = subprocess.run([sys.executable, "-c", code], cwd=Path(__file__).resolve().parents[1],
                         capture_output=True, text=True)
    assert got.returncode == 0, got.stderr
