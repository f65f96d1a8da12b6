"""The attention's workspace is checked and used under one plan (host).

The library's own device query and launchers are stood in for by a shared object
loaded before it: the multiprocessor count changes between the size query and the
launch (as it did where the first call of a process cached the real count), and the
launchers note the plans they were given."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STAND_IN = r"""
#include "kernels.h"
#include <string.h>
namespace qlin {
static int sms = 152, later = 152;
static size_t used;
static char *base;
static DeviceInfo dev;
int sm_count() { return sms; }
qlin_status current_device(DeviceInfo **out) {
  sms = later;
  dev.device = 0, dev.sms = sms, dev.cc_major = 10, dev.cc_minor = 3;
  *out = &dev;
  return QLIN_OK;
}
static void use(void *ws, size_t bytes) {
  const size_t end = ws ? (size_t)((char *)ws - base) + bytes : 0;
  if (end > used) used = end;
}
cudaError_t launch_attn_split(const AttnArgs &, const AttnSplitPlan &plan, int, void *ws, unsigned *, cudaStream_t) {
  use(ws, plan.ws_bytes);
  return cudaSuccess;
}
cudaError_t launch_attn_prefill(const AttnArgs &, const AttnPrefillPlan &plan, int, void *ws, unsigned *,
                                cudaStream_t) {
  use(ws, plan.ws_bytes);
  return cudaSuccess;
}
}  // namespace qlin
extern "C" void stand_in_reset(int first, int then, void *ws) {
  qlin::sms = first, qlin::later = then, qlin::used = 0, qlin::base = (char *)ws;
}
extern "C" size_t stand_in_used() { return qlin::used; }
"""

PROBE = r"""
import ctypes, sys
s = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
s.stand_in_used.restype = ctypes.c_size_t
sys.path.insert(0, sys.argv[2])
from bit_quantized_linear_gb300 import capi
L, P = capi.lib(), ctypes.c_void_p
G, WS = P(4096), 1 << 20
bad = seen = 0
for B, Hq, H in [(1, 28, 4), (3, 16, 2), (8, 8, 8), (64, 32, 8)]:
    for D in (64, 128, 256):
        for q in (1, 40, 200, 1000):
            for kv in (300, 2048, 8192, 32768):
                for then in (132, 148, 160, 188):
                    s.stand_in_reset(152, then, P(WS))
                    need = capi.qlin_attn_mixed_workspace_bytes(B, Hq, H, D, q, kv, 0)
                    st = L.qlin_attn_mixed(B, B * q, Hq, H, D, G, Hq * D, G, q, G, kv, G, 2048, 16, 32768, G, G, G, G,
                                           0.1, 1, 0, G, Hq * D, P(WS) if need else None, need, None)
                    assert st == capi.QLIN_OK, (st, B, Hq, H, D, q, kv)
                    seen += s.stand_in_used() > 0
                    if s.stand_in_used() > need:
                        bad += 1
                        print("beyond", B, Hq, H, D, q, kv, then, need, s.stand_in_used())
print("seen", seen, "bad", bad)
sys.exit(1 if bad or not seen else 0)
"""


def test_launch_stays_within_the_checked_size(tmp_path):
    from bit_quantized_linear_gb300 import build
    build.build()
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("needs g++")
    src, so = tmp_path / "stand_in.cc", tmp_path / "stand_in.so"
    src.write_text(STAND_IN)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", f"-I{cuda}", f"-I{build.CSRC}", f"-I{build.INCLUDE}",
                    str(src), "-o", str(so)], check=True, capture_output=True, text=True)
    r = subprocess.run([sys.executable, "-c", PROBE, str(so), ROOT], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
