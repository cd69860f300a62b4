"""The operators around a linear layer: their host code under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only), driven through argument checks that end before a HIP
call, with sizes and strides up to the ends of their types (sums and products of them must not
leave 64 bits, whatever a caller passes)."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

DRIVER = r"""
#include <math.h>
#include <stdio.h>
#include "kq.h"

static int fails = 0, calls = 0;
#define CHECK(c) do { ++calls; if (!(c)) { printf("FAIL line %d: %s\n", __LINE__, #c); ++fails; } } while (0)
#define P(a) ((void *)(uintptr_t)(a))
static const int64_t big[] = {-(1ll << 62) - 1, -1, 0, 1, 7, 8, 64, 4096, 65536, 1 << 20, (1ll << 31) - 1, 1ll << 31,
                              1ll << 40, (1ll << 48) + 16, 1ll << 62, 0x7FFFFFFFFFFFFFFFll};
#define EACH(i) for (unsigned i = 0; i < sizeof(big) / sizeof(big[0]); ++i)

/* no address: a call that gets past the sizes is refused for its NULLs, or has no rows to work on */
int main(void) {
  size_t bytes = 0;
  EACH(i) EACH(j) EACH(k) {
    const int64_t a = big[i], b = big[j], c = big[k];
    kq_status st = kq_rmsnorm_quant(NULL, c, NULL, c, NULL, a, b, KQ_BF16, 1e-5f, 1.f, KQ_FP16, NULL, c, NULL, c,
                                    NULL, NULL, NULL);
    CHECK(st != KQ_OK || a == 0);
    st = kq_grouped_gemm(NULL, c, NULL, a, NULL, b, NULL, c, c, NULL, a, c, b, NULL, 4, KQ_FP16, KQ_BF16, NULL, c,
                         NULL);
    CHECK(st != KQ_OK || a == 0 || b == 0);
    st = kq_adapter_add(NULL, c, NULL, NULL, NULL, NULL, NULL, c, a, b, c, 16, a, KQ_BF16, NULL, c, NULL, 0, NULL);
    CHECK(st != KQ_OK || a == 0 || c == 0);
    st = kq_adapter_workspace_size(a, b, c, &bytes);
    CHECK(st != KQ_OK || (a >= 0 && b > 0 && c > 0 && bytes < (1ull << 40)));
    /* with addresses, all in one place: strides, spans and overlaps are worked out, and refused */
    st = kq_rmsnorm_quant(P(4096), c, P(4096), b, P(4096), a, 64, KQ_FP32, 1e-5f, 1.f, KQ_FP32, P(4096), c, P(4096),
                          b, P(4096), P(4096), NULL);
    CHECK(st != KQ_OK || a == 0);
    st = kq_grouped_gemm(P(4096), c, P(4096), a < 0 ? a : 8, P(4096), a, P(4096), b, c, P(4096), b, 256, 4, P(4096), 8,
                         KQ_FP32, KQ_FP32, P(4096), c, NULL);
    CHECK(st != KQ_OK || a == 0 || b == 0);
    st = kq_adapter_add(P(4096), c, P(4096), P(4096), P(4096), P(4096), P(4096), b, a, 64, 64, 16, c, KQ_BF16, P(4096),
                        b, P(4096), ~(size_t)0, NULL);
    CHECK(st != KQ_OK || a == 0);
  }
  CHECK(kq_adapter_workspace_size(8, 64, 16, NULL) == KQ_ERR_INVALID_ARG);
  CHECK(kq_rmsnorm_quant(P(4096), 64, NULL, 0, P(8192), 1, 64, (kq_dtype)77, 0.f, 1.f, KQ_FP16, NULL, 0, NULL, 0,
                         P(16384), P(32768), NULL) == KQ_ERR_INVALID_ARG);
  CHECK(kq_rmsnorm_quant(P(4096), 64, NULL, 0, P(8192), 1, 64, KQ_BF16, 0.f, NAN, KQ_FP16, NULL, 0, NULL, 0, P(16384),
                         P(32768), NULL) == KQ_ERR_INVALID_ARG);
  CHECK(kq_rmsnorm_quant(P(4097), 64, NULL, 0, P(8192), 1, 64, KQ_BF16, 0.f, 1.f, KQ_FP16, NULL, 0, NULL, 0, P(16384),
                         P(32768), NULL) == KQ_ERR_ALIGNMENT);
  CHECK(kq_adapter_add(P(4096), 64, P(65536), P(131072), P(262144), NULL, NULL, 0, 4, 64, 64, 16, 2, KQ_FP16,
                       P(524288), 64, P(1048576), 255, NULL) == KQ_ERR_WORKSPACE);
  printf("%d host checks done, %d failed\n", calls, fails);
  return fails != 0;
}
"""


def test_host_code_under_address_and_undefined_behaviour_sanitizers(tmp_path):
    H = pytest.importorskip("test_host_sanitizers")  # how the sources are compiled
    if not (os.path.exists(H.HIPCC) and os.path.exists(H.CLANG) and os.path.exists(H.CLANGXX)):
        pytest.skip("ROCm compilers not available")
    from kronecker_factored_transforms_amd import binding as B
    B.lib()  # the other sources come from the library
    srcs = ["kq_norm", "kq_grouped", "kq_adapter"]
    objs = [str(tmp_path / (s + ".o")) for s in srcs]
    with ThreadPoolExecutor(len(srcs)) as ex:
        list(ex.map(H._host_sanitized_compile, [os.path.join(H.CSRC, s + ".hip") for s in srcs], objs))
    drv = tmp_path / "driver.c"
    drv.write_text(DRIVER)
    sanitize = ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined"]
    r = subprocess.run([H.CLANG, "-std=gnu99", "-O1", "-g", "-Wall", "-Werror", *sanitize, "-I",
                        os.path.join(H.ROOT, "include"), "-c", str(drv), "-o", str(tmp_path / "driver.o")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    exe, where = str(tmp_path / "driver"), os.path.dirname(B.LIB_PATH)
    r = subprocess.run([H.CLANGXX, *sanitize, str(tmp_path / "driver.o"), *objs, "-o", exe, "-L", where, "-lkq",
                        "-L", os.path.join(H.ROCM, "lib"), "-lamdhip64",
                        f"-Wl,-rpath,{where}:{os.path.join(H.ROCM, 'lib')}"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    env.pop("KQ_LOG", None)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and "host checks done, 0 failed" in r.stdout, (r.stdout[-3000:], r.stderr[-3000:])
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr
