"""The host checks of the tensor-list and 4-bit entry points under the host
sanitizers (CPU only): the same build as test_host_sanitizers, with a driver that
fills tables for many lists, in buffers of exactly the asked size, and walks the
refusals of each entry point."""
import glob
import os
import subprocess

import pytest

DRIVER = r'''
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <memory>
#include <vector>
#include "iqlher.h"
static int failures = 0;
#define EXPECT(call, code) do { int rc_ = (call); if (rc_ != (code)) { \
    std::printf("line %d: %s returned %d, expected %d (%s)\n", __LINE__, #call, rc_, (int)(code), iqlh_last_error()); \
    ++failures; } else if ((code) != IQLH_OK && iqlh_last_error()[0] == 0) { \
    std::printf("line %d: no error message\n", __LINE__); ++failures; } } while (0)
struct Piece { uint64_t ptr; int64_t off; int32_t n, dtype, r[2]; };
int main() {
    uint32_t seed = 1;
    auto rnd = [&](uint32_t n) { seed = seed * 1664525u + 1013904223u; return (seed >> 8) % n; };
    for (int rep = 0; rep < 300; ++rep) {
        const int count = 1 + rnd(rep < 200 ? 20 : 400);
        std::vector<int64_t> lens(count);
        std::vector<int32_t> types(count);
        std::vector<const void*> ptrs(count);
        uint64_t at = 1 << 20;
        for (int i = 0; i < count; ++i) {
            types[i] = rnd(3);
            const int es = types[i] == IQLH_F32 ? 4 : 2;
            lens[i] = rnd(4) == 0 ? rnd(3) : rnd(rep % 2 ? 200000 : 3000);
            at += 4 + es * rnd(9);
            at -= at % es;
            ptrs[i] = lens[i] ? (const void*)at : nullptr;
            at += lens[i] * es;
        }
        size_t bytes = 0;
        EXPECT(iqlh_tensor_set_bytes(lens.data(), types.data(), count, &bytes), IQLH_OK);
        char* table = (char*)std::aligned_alloc(16, (bytes + 15) / 16 * 16);
        iqlh_tensor_set set;
        EXPECT(iqlh_tensor_set_fill(ptrs.data(), lens.data(), types.data(), count, table, bytes, &set), IQLH_OK);
        if (set.table_bytes > bytes) { std::printf("table too long\n"); ++failures; }
        int64_t sum = 0;
        for (int k = 0; k < set.pieces; ++k) {
            Piece p; std::memcpy(&p, table + sizeof(p) * k, sizeof(p));
            if (p.off != sum || p.n < 1) ++failures;
            sum += p.n;
        }
        if (sum != set.numel) { std::printf("pieces cover %lld of %lld\n", (long long)sum, (long long)set.numel); ++failures; }
        int32_t last = 0; std::memcpy(&last, table + sizeof(Piece) * set.pieces + 4 * count, 4);
        if (last != set.pieces) ++failures;
        size_t ws = 0;
        EXPECT(iqlh_grad_norm_workspace_bytes(&set, &ws), IQLH_OK);
        EXPECT(iqlh_grad_norm(&set, IQLH_NORM_L2, (float*)16, nullptr, nullptr, (void*)16, ws, nullptr), IQLH_EINVAL);
        set.d_table = (void*)4096;
        EXPECT(iqlh_grad_norm(&set, 7, (float*)16, nullptr, nullptr, (void*)16, ws, nullptr), IQLH_EINVAL);
        EXPECT(iqlh_grad_clip(&set, 0, NAN, nullptr, (float*)16, nullptr, (void*)16, ws, nullptr), IQLH_EINVAL);
        EXPECT(iqlh_grad_clip(&set, 0, 1.f, nullptr, (float*)16, nullptr, (void*)16, ws - 1, nullptr), IQLH_EINVAL);
        std::free(table);
    }
    int64_t big[3] = {(int64_t)1 << 40, (int64_t)1 << 40, INT64_MAX};
    int32_t f32[3] = {0, 0, 0};
    size_t bytes = 0;
    EXPECT(iqlh_tensor_set_bytes(big, f32, 3, &bytes), IQLH_EINVAL);
    EXPECT(iqlh_tensor_set_bytes(big, f32, -1, &bytes), IQLH_EINVAL);
    EXPECT(iqlh_tensor_set_bytes(big, f32, 2, &bytes), IQLH_OK);
    iqlh_mx4 q = {(uint8_t*)4096, (uint8_t*)4096, 64, 64};
    EXPECT(iqlh_mx4_quantize(nullptr, 0, 64, 0, &q, nullptr), IQLH_EINVAL);
    EXPECT(iqlh_mx4_quantize((void*)16, 0, INT64_MAX, 0, &q, nullptr), IQLH_EINVAL);
    EXPECT(iqlh_mx4_dequantize(&q, (void*)16, 9, 64, nullptr), IQLH_EINVAL);
    EXPECT(iqlh_mx4_workspace_bytes((int64_t)1 << 30, (int64_t)1 << 30, (int64_t)1 << 30, &bytes), IQLH_OK);
    EXPECT(iqlh_mx4_workspace_bytes(INT64_MAX, 1, 1, &bytes), IQLH_EINVAL);
    for (int64_t m : {1, 16, 17, 500, 5000, 70000}) for (int64_t n : {1, 300, 9000}) for (int64_t k : {1, 33, 600, 1 << 20}) {
        size_t need = 0;
        EXPECT(iqlh_mx4_workspace_bytes(m, n, k, &need), IQLH_OK);
        iqlh_mx4 a = {(uint8_t*)4096, (uint8_t*)4096, m, k}, b = {(uint8_t*)4096, (uint8_t*)4096, n, k};
        EXPECT(iqlh_mx4_matmul(&a, &b, nullptr, 0, (void*)16, 0, n, (void*)16, need - 1, nullptr), IQLH_EINVAL);
        EXPECT(iqlh_mx4_linear((void*)16, 1, k, m, &b, nullptr, 0, (void*)16, 0, n - 1, (void*)16, need, nullptr), IQLH_EINVAL);
    }
    EXPECT(iql_forward_values_mx4_workspace_bytes(nullptr, 1, &bytes), IQLH_EINVAL);
    EXPECT(iql_forward_values_mx4(nullptr, (void*)16, 0, 4, 1, (float*)16, nullptr, nullptr, 0.9f, nullptr, (void*)16, 64,
                                  nullptr), IQLH_EINVAL);
    std::printf("%d failures\n", failures);
    return failures == 0 ? 0 : 1;
}
'''


def test_new_entry_points_are_clean_under_the_host_sanitizers(tmp_path):
    base = pytest.importorskip("tests.test_host_sanitizers")
    if not os.path.exists(base.HIPCC):
        pytest.skip("hipcc not available")
    objs = [o for o in sorted(glob.glob(os.path.join(base.ROOT, "offline_rl_step_amd", "_build", "*.o")))
            if not o.endswith("api.hip.o")]
    if len(objs) < 5:
        pytest.skip("library objects not built (python offline_rl_step_amd/build.py)")
    drv = tmp_path / "driver.hip"
    drv.write_text(DRIVER)
    outs = []
    for src in (os.path.join(base.ROOT, "offline_rl_step_amd", "csrc", "api.hip"), str(drv)):
        out = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([base.HIPCC, *base.FLAGS, *base.SAN, "-c", src, "-o", out], capture_output=True, text=True)
        assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
        outs.append(out)
    exe = str(tmp_path / "driver")
    r = subprocess.run([base.HIPCC, "--offload-arch=gfx950", *base.SAN, *outs, *objs, "-o", exe], capture_output=True,
                       text=True)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    text = r.stdout + r.stderr
    assert "ERROR: AddressSanitizer" not in text and "runtime error" not in text, text[-4000:]
    assert r.returncode == 0 and "0 failures" in r.stdout, text[-4000:]
