"""Where a call's scratch lies in a workspace that is only 16-byte aligned (a slice of a caller's arena): the partial
rows that the kernels write in 32-byte stores must start on 32 bytes, and everything must end inside the workspace.
A host program built from the library's own headers prints the addresses; nothing is launched."""
import os
import subprocess

import pytest

from prefix_shared_kv_ra_gb300 import _build

PROBE = r"""
#include <cstdio>
#include "decode_internal.h"
#include "tree_internal.h"

using namespace ra;

static void at(const char* what, uint8_t* ws, size_t total, const void* p, size_t bytes) {
  const uint8_t* b = static_cast<const uint8_t*>(p);
  std::printf("%s %d %d\n", what, static_cast<int>(reinterpret_cast<uintptr_t>(p) % 32),
              b >= ws && b + bytes <= ws + total ? 1 : 0);
}

int main() {
  for (int shift = 0; shift < 32; shift += 16) {
    uint8_t* ws = reinterpret_cast<uint8_t*>((uintptr_t(1) << 32) + shift);
    for (int batch : {1, 34, 64, 98})
      for (int groups : {0, 2}) {
        const int hq = 32, hkv = 8, d = 128;
        const DecodePlan pl = plan_decode(batch, hq, hkv, d, 4096, groups, groups ? 1024 : 0, groups ? 1 : 0);
        const DecodeWorkspace wl = layout_decode_workspace(batch, hq, hkv, d, pl, groups ? 1 : 0);
        DecodeParams p{};
        p.batch = batch;
        bind_decode_workspace(p, wl, pl, ws);
        at("decode_part_o", ws, wl.total, p.part_o, size_t(pl.max_items) * hq * d * 4);
        at("decode_part_lse", ws, wl.total, p.part_lse, size_t(pl.max_items) * hq * 4);
        if (groups) at("decode_casc_o", ws, wl.total, p.casc_o, size_t(batch) * hq * pl.max_csplits * d * 4);
        if (groups) at("decode_casc_lse", ws, wl.total, p.casc_lse, size_t(batch) * hq * pl.max_csplits * 4);
        at("decode_ints", ws, wl.total, p.req_done, size_t(batch) * 4);
      }
    for (int draft : {1, 8, 16, 32, 64, 1024})
      for (int tiled : {0, 1}) {
        const int hq = 32, hkv = 8, d = 64, batch = 7, total_q = 200;
        if (tiled && !tree_tileable(hq, hkv, draft)) continue;
        const TreeShape sh = tree_shape(hq, hkv, d, draft, tiled);
        const size_t total = layout_tree(batch, total_q, hq, hkv, d, draft, sh, nullptr).total;
        const TreeWorkspace w = layout_tree(batch, total_q, hq, hkv, d, draft, sh, ws);
        const size_t rows = size_t(w.cap_parts) * hkv * w.part_rows;
        at("tree_header", ws, total, w.header, 32);
        at("tree_items", ws, total, w.items, size_t(w.cap) * 32);
        at("tree_merges", ws, total, w.merges, size_t(w.cap_parts) * 16);
        at("tree_bad", ws, total, w.bad, size_t(w.cap_parts > batch ? w.cap_parts : batch) * hkv * 4);
        at("tree_part_lse", ws, total, w.part_lse, rows * 4);
        at("tree_part_o", ws, total, w.part_o, rows * d * 4);
      }
  }
}
"""


@pytest.fixture(scope="module")
def sections(tmp_path_factory):
    lib = _build.build()
    at = tmp_path_factory.mktemp("probe")
    src, exe = at / "probe.cu", at / "probe"
    src.write_text(PROBE)
    r = subprocess.run([_build._nvcc(), *_build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I",
                        os.path.join(_build.ROOT, "include"), "-I", _build.CSRC, str(src), lib, "-o", str(exe),
                        "-Xlinker", f"-rpath={os.path.dirname(lib)}"], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    return [(name, int(mod), int(inside)) for name, mod, inside in (line.split() for line in out.splitlines())]


def test_partial_rows_start_on_32_bytes(sections):
    rows = [s for s in sections if s[0] in ("decode_part_o", "decode_casc_o", "tree_part_o")]
    assert {s[0] for s in rows} == {"decode_part_o", "decode_casc_o", "tree_part_o"}
    assert [s for s in rows if s[1] != 0] == []


def test_sections_end_inside_the_workspace(sections):
    assert [s for s in sections if s[2] != 1] == []
    assert [s for s in sections if s[1] % 4 != 0] == []
