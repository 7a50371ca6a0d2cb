"""The policy loss's and the matrix sets' host code under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only):
tables of random lists, written into heap blocks of exactly the size asked for, and the refusals of every entry point,
each before its first HIP call.  Built as in test_host_sanitizers.py, whose flags it takes."""
import glob
import os
import subprocess

import pytest

base = pytest.importorskip("tests.test_host_sanitizers")

DRIVER = r'''
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>
#include "iqlher.h"
static int failures = 0;
#define EXPECT(call, code) do { int rc_ = (call); if (rc_ != (code)) { \
    std::printf("line %d: %s returned %d, expected %d (%s)\n", __LINE__, #call, rc_, (int)(code), iqlh_last_error()); \
    ++failures; } else if ((code) != IQLH_OK && iqlh_last_error()[0] == 0) { \
    std::printf("line %d: no error message\n", __LINE__); ++failures; } } while (0)
static const int64_t kBase = (int64_t)1 << 40;
static iqlh_matrix matrix(int64_t rows, int64_t cols, int i, bool momentum) {
    iqlh_matrix m; std::memset(&m, 0, sizeof(m));
    const int64_t at = kBase * (1 + 3 * (int64_t)i);
    m.x = (void*)at; m.out = (void*)(at + kBase); m.momentum = momentum ? (float*)(at + 2 * kBase) : nullptr;
    m.rows = rows; m.cols = cols; m.ld_x = m.ld_out = m.ld_momentum = cols;
    m.x_dtype = IQLH_BF16; m.out_dtype = i % 2 ? IQLH_F32 : IQLH_BF16; m.compute_dtype = i % 2 ? IQLH_F32 : IQLH_F16;
    return m;
}
static int fill(std::vector<iqlh_matrix>& ms, iqlh_matrix_set* set, size_t short_by) {
    size_t bytes = 0;
    int rc = iqlh_matrix_set_bytes(ms.data(), (int32_t)ms.size(), &bytes);
    if (rc) return rc;
    void* host = std::aligned_alloc(16, (bytes + 15) / 16 * 16);
    std::memset(host, 0xFF, bytes);
    rc = iqlh_matrix_set_fill(ms.data(), (int32_t)ms.size(), host, bytes - short_by, set);
    if (rc == IQLH_OK && set->table_bytes > bytes) { std::printf("table above its size\n"); ++failures; }
    std::free(host);
    return rc;
}
int main() {
    std::mt19937_64 g(7);
    auto size = [&](double top) { return (int64_t)std::exp(std::uniform_real_distribution<double>(0.0, std::log(top))(g)); };
    iqlh_matrix_set set;
    for (int rep = 0; rep < 60; ++rep) {
        std::vector<iqlh_matrix> ms;
        const int n = rep < 40 ? 1 + (int)(g() % 12) : 200 + (int)(g() % 200);
        for (int i = 0; i < n; ++i) ms.push_back(matrix(size(rep < 40 ? 9000 : 400), size(rep < 40 ? 9000 : 400), i, rep % 2));
        EXPECT(fill(ms, &set, 0), IQLH_OK);
        EXPECT(fill(ms, &set, 1), IQLH_EINVAL);
    }
    std::vector<iqlh_matrix> most;
    for (int i = 0; i < 4096; ++i) most.push_back(matrix(1 + i % 300, 1 + i % 70, i, true));
    EXPECT(fill(most, &set, 0), IQLH_OK);
    std::vector<iqlh_matrix> large{matrix(65536, 65536, 0, true), matrix(65536, 1, 1, true), matrix(1, 65536, 2, true)};
    EXPECT(fill(large, &set, 0), IQLH_OK);
    large.assign(20, large[0]);
    EXPECT(iqlh_matrix_set_bytes(large.data(), 20, nullptr), IQLH_EINVAL);
    size_t bytes = 0;
    EXPECT(iqlh_matrix_set_bytes(large.data(), 20, &bytes), IQLH_ESHAPE);  // more tiles than one launch takes
    EXPECT(iqlh_matrix_set_bytes(nullptr, 1, &bytes), IQLH_EINVAL);
    EXPECT(iqlh_matrix_set_bytes(most.data(), 4097, &bytes), IQLH_EINVAL);
    EXPECT(iqlh_matrix_set_bytes(most.data(), -1, &bytes), IQLH_EINVAL);
    std::vector<iqlh_matrix> two{matrix(30, 40, 0, true), matrix(50, 20, 1, true)};
    EXPECT(iqlh_matrix_set_fill(two.data(), 2, nullptr, 1 << 20, &set), IQLH_EINVAL);
    two[1].x = nullptr;
    EXPECT(fill(two, &set, 0), IQLH_EINVAL);
    two[1] = matrix(50, 20, 1, false);
    EXPECT(fill(two, &set, 0), IQLH_EINVAL);
    two[1] = matrix(50, 20, 0, true);
    EXPECT(fill(two, &set, 0), IQLH_EINVAL);  // shares memory
    two[1] = matrix(50, 20, 1, true);
    two[1].ld_out = 19;
    EXPECT(fill(two, &set, 0), IQLH_EINVAL);
    two[1].ld_out = INT64_MAX;
    EXPECT(fill(two, &set, 0), IQLH_EINVAL);
    two[1].ld_out = 20, two[1].rows = INT64_MAX;
    EXPECT(fill(two, &set, 0), IQLH_ESHAPE);
    two[1].rows = 50, two[1].x = (void*)(UINTPTR_MAX - 63);  // ends behind the last address
    (void)fill(two, &set, 0);
    // the calls
    two[1] = matrix(50, 20, 1, true);
    EXPECT(fill(two, &set, 0), IQLH_OK);
    void* p = (void*)kBase;
    EXPECT(iqlh_orthogonalize(nullptr, 5, 1e-7, nullptr, p, 1 << 30, nullptr), IQLH_EINVAL);
    EXPECT(iqlh_orthogonalize(&set, 5, 1e-7, nullptr, p, 1 << 30, nullptr), IQLH_EINVAL);  // no table
    set.d_table = p;
    EXPECT(iqlh_orthogonalize(&set, 33, 1e-7, nullptr, p, 1 << 30, nullptr), IQLH_EINVAL);
    EXPECT(iqlh_orthogonalize(&set, 5, NAN, nullptr, p, 1 << 30, nullptr), IQLH_EINVAL);
    EXPECT(iqlh_orthogonalize(&set, 5, 1e-7, nullptr, nullptr, 1 << 30, nullptr), IQLH_EINVAL);
    EXPECT(iqlh_orthogonalize(&set, 5, 1e-7, nullptr, p, set.workspace_bytes - 1, nullptr), IQLH_EINVAL);
    const double values[] = {NAN, INFINITY, -INFINITY, 1e308, -1e308};
    for (double v : values) {
        EXPECT(iqlh_muon_step(&set, v, 0.9, 1, 0.1, 0, 5, 1e-7, nullptr, p, 1 << 30, nullptr), IQLH_EINVAL);
        EXPECT(iqlh_muon_step(&set, 0.1, v, 1, 0.1, 0, 5, 1e-7, nullptr, p, 1 << 30, nullptr), IQLH_EINVAL);
        EXPECT(iqlh_muon_step(&set, 0.1, 0.9, 1, v, 0, 5, 1e-7, nullptr, p, 1 << 30, nullptr), IQLH_EINVAL);
    }
    EXPECT(iqlh_muon_step(&set, 0.1, 0.9, 2, 0.1, 0, 5, 1e-7, nullptr, p, 1 << 30, nullptr), IQLH_EINVAL);
    EXPECT(iqlh_muon_step(&set, 0.1, 0.9, 1, 0.1, 9, 5, 1e-7, nullptr, p, 1 << 30, nullptr), IQLH_EINVAL);
    // policy loss: sizes over the whole range, then refusals
    for (int rep = 0; rep < 3000; ++rep) {
        const int64_t rows = size(1 << 24), actions = size(1 << 24), dim = size(1 << 14), top = (int64_t)1 << 38;
        const bool fits = rows * actions <= top && rows * dim <= top && actions * dim <= top;
        for (int t : {IQLH_F32, IQLH_BF16, IQLH_F16})
            for (int grad = 0; grad < 2; ++grad) EXPECT(iqlh_policy_loss_workspace_bytes(rows, actions, dim, t, grad, &bytes), fits ? IQLH_OK : IQLH_ESHAPE);
    }
    const int64_t bad[] = {0, -1, INT64_MIN, INT64_MAX, ((int64_t)1 << 24) + 1};
    for (int64_t b : bad)
        for (int k = 0; k < 3; ++k)
            EXPECT(iqlh_policy_loss_workspace_bytes(k == 0 ? b : 4, k == 1 ? b : 4, k == 2 ? b : 4, IQLH_F32, 1, &bytes), IQLH_ESHAPE);
    EXPECT(iqlh_policy_loss_workspace_bytes(4, 4, 4, 9, 1, &bytes), IQLH_EINVAL);
    EXPECT(iqlh_policy_loss_workspace_bytes(4, 4, 4, IQLH_F32, 2, &bytes), IQLH_EINVAL);
    EXPECT(iqlh_policy_loss_workspace_bytes(4, 4, 4, IQLH_F32, 1, nullptr), IQLH_EINVAL);
    iqlh_policy_head head; std::memset(&head, 0, sizeof(head));
    head.hidden = (void*)kBase; head.weight = (void*)(2 * kBase); head.rows = 16; head.actions = 100; head.dim = 8;
    head.ld_hidden = head.ld_weight = 8; head.dtype = IQLH_BF16;
    auto at = [&](int i) { return (float*)(i * kBase); };
    auto loss = [&](const iqlh_policy_head* h, double scale, float* nll, size_t wb) {
        return iqlh_policy_loss(h, (int32_t*)at(3), nullptr, scale, nll, at(5), at(6), nullptr, at(7), wb, nullptr);
    };
    auto grad = [&](const iqlh_policy_head* h, double scale, int64_t ld, size_t wb) {
        return iqlh_policy_loss_grad(h, (int32_t*)at(3), nullptr, scale, at(5), at(8), ld, at(9), 8, at(10), at(7), wb, nullptr);
    };
    EXPECT(loss(nullptr, 1.0, at(4), 1 << 30), IQLH_EINVAL);
    EXPECT(grad(nullptr, 1.0, 8, 1 << 30), IQLH_EINVAL);
    for (double v : values) {
        EXPECT(loss(&head, v, at(4), 1 << 30), IQLH_EINVAL);
        EXPECT(grad(&head, v, 8, 1 << 30), IQLH_EINVAL);
    }
    EXPECT(loss(&head, 1.0, nullptr, 1 << 30), IQLH_EINVAL);
    EXPECT(loss(&head, 1.0, at(5), 1 << 30), IQLH_EINVAL);
    EXPECT(loss(&head, 1.0, at(4), 8), IQLH_EINVAL);
    EXPECT(grad(&head, 1.0, 7, 1 << 30), IQLH_EINVAL);
    EXPECT(grad(&head, 1.0, INT64_MIN, 1 << 30), IQLH_EINVAL);
    EXPECT(grad(&head, 1.0, 8, 8), IQLH_EINVAL);
    head.ld_weight = INT64_MAX;
    EXPECT(grad(&head, 1.0, 8, 8), IQLH_EINVAL);
    EXPECT(loss(&head, 1.0, at(4), 8), IQLH_EINVAL);
    std::printf("%d failures\n", failures);
    return failures == 0 ? 0 : 1;
}
'''


def test_lists_and_refusals_are_clean_under_asan_and_ubsan(tmp_path):
    if not os.path.exists(base.HIPCC):
        pytest.skip("hipcc not available")
    objs = [o for o in sorted(glob.glob(os.path.join(base.ROOT, "offline_rl_step_amd", "_build", "*.o")))
            if not o.endswith("api.hip.o")]
    if len(objs) < 5:
        pytest.skip("library objects not built (python offline_rl_step_amd/build.py)")
    source = tmp_path / "driver.hip"
    source.write_text(DRIVER)
    parts = []
    for name in (os.path.join(base.ROOT, "offline_rl_step_amd", "csrc", "api.hip"), str(source)):
        parts.append(str(tmp_path / (os.path.basename(name) + ".o")))
        r = subprocess.run([base.HIPCC, *base.FLAGS, *base.SAN, "-c", name, "-o", parts[-1]], capture_output=True, text=True)
        assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    exe = str(tmp_path / "driver")
    r = subprocess.run([base.HIPCC, "--offload-arch=gfx950", *base.SAN, *parts, *objs, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    out = r.stdout + r.stderr
    assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert r.returncode == 0 and "0 failures" in r.stdout, out[-4000:]
