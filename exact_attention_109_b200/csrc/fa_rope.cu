// fa_rope.cu -- C entry points of the passes before attention: norm and
// rotation of queries and keys with its gradient, and appending to a paged
// cache (declared in include/fa.h; kernels in fa_rope_kernels.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "fa.h"
#include "fa_internal.h"
#include "fa_rope_kernels.cuh"

namespace {

using fa_host::aligned;

// CTAs of the backward kernel at most, and so rows of its dw partials in the
// workspace: two waves of the two that an SM's registers hold, on 148 SMs.
constexpr int kBwdCtasPerSm = 2;
constexpr int kMaxBwdCtas = 592;
constexpr long long kMinHeads = 2;    // heads that a CTA takes at least
constexpr long long kManyHeads = 16;  // from twice that in one wave on, CTAs take half each:
                                      // the second wave evens out the first (16384 tokens of
                                      // 48 heads of 128: 102 -> 100 us)
// CTAs of the forward kernel that an SM holds: up to one wave of them, the heads
// of a token block are spread over more CTAs.
constexpr int kPrepCtasPerSm = 3;
constexpr int kHeadsPerCta = 16;

// Strides (in elements) of one input tensor: 16-byte rows, no negative step.
bool strides_ok(const long long* s, int n) {
    for (int i = 0; i < n; ++i)
        if (s[i] < 0 || s[i] % 8 != 0 || s[i] > (1ll << 40)) return false;
    return true;
}

// The rows of an output [n0][n1][n2] of `d` values must not overlap: taken by
// rising stride, each dimension steps over all of the ones before it.
bool disjoint_rows(const long long* s, long long n0, long long n1, long long n2, int d) {
    long long st[3] = {s[0], s[1], s[2]}, n[3] = {n0, n1, n2};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (st[j] < st[i]) std::swap(st[i], st[j]), std::swap(n[i], n[j]);
    long long extent = d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (st[i] < extent) return false;
        if (n[i] - 1 > ((1ll << 62) - extent) / std::max(1ll, st[i])) return false;
        extent += (n[i] - 1) * st[i];
    }
    return true;
}

fa_status check_heads(int Hq, int Hkv, int d) {
    if (Hq < 1 || Hkv < 1 || Hq > (1 << 16) || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
    return d == 64 || d == 128 ? FA_OK : FA_ERR_UNSUPPORTED;
}

// Norm weights and rotation: both weights or none; a table of at least one
// row whose width is a multiple of 16 up to d, or none; one of the two.
fa_status check_norm_rope(const void* wq, const void* wk, int w_f32, float eps,
                          const float* rope, long long rows, int rope_dim, int d) {
    if ((wq == nullptr) != (wk == nullptr)) return FA_ERR_INVALID_ARG;
    if (wq && !(std::isfinite(eps) && eps > 0.f)) return FA_ERR_INVALID_ARG;
    if (w_f32 != 0 && w_f32 != 1) return FA_ERR_INVALID_ARG;
    const uintptr_t wb = w_f32 ? 4 : 2;
    if (!aligned(wq, wb) || !aligned(wk, wb)) return FA_ERR_MISALIGNED;
    if (rope) {
        if (rows < 1 || rows > (1ll << 40) || rope_dim < 16 || rope_dim > d || rope_dim % 16)
            return FA_ERR_INVALID_ARG;
        if (!aligned(rope, 16)) return FA_ERR_MISALIGNED;
    }
    return FA_OK;
}

fa::RopeParams rope_params(const void* wq, const void* wk, int w_f32, float eps,
                           const float* rope, long long rows, int rope_dim, const int* positions,
                           int B, int N, int Hq, int Hkv, unsigned int* err) {
    fa::RopeParams p;
    p.table = reinterpret_cast<const float2*>(rope);
    p.rows = rows;
    p.rope_dim = rope ? rope_dim : 0;
    p.positions = positions;
    p.wq = wq;
    p.wk = wk;
    p.w_f32 = w_f32;
    p.eps = eps;
    p.B = B;
    p.N = N;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.heads_per_cta = 0;
    p.err = err;
    return p;
}

// Groups the heads are cut into: enough CTAs to fill the SMs, and no more
// than about 16 heads for one.  16384 tokens of 48 heads of 128: 73 us with all
// heads in a CTA, 69.5 with 24, 68 with 16 (the last wave is shorter), 77 with
// 10 (the set-up of a CTA counts).
int head_groups(long long blocks, int heads, int sms) {
    const long long g =
        std::max<long long>(1ll * kPrepCtasPerSm * sms / blocks, heads / kHeadsPerCta);
    return static_cast<int>(std::max(1ll, std::min<long long>(g, heads)));
}

template <int D, bool IL, bool PAGED>
cudaError_t launch_prep(const fa::HeadRows& q, const fa::HeadRows& k, const fa::HeadRows& v,
                        fa::RopeParams p, const fa::PrepOut& out, const fa::PagedDest& dst,
                        int sms, cudaStream_t s) {
    constexpr int TOKENS = fa::kRopeThreads / (D / 8);
    const long long blocks = (static_cast<long long>(p.B) * p.N + TOKENS - 1) / TOKENS;
    const int heads = p.Hq + p.Hkv + (v.p ? p.Hkv : 0);
    const int groups = head_groups(blocks, heads, sms);
    p.heads_per_cta = (heads + groups - 1) / groups;
    const dim3 grid(static_cast<unsigned>(blocks), (heads + p.heads_per_cta - 1) / p.heads_per_cta);
    return fa_host::launch_overlapped(fa::fa_prep_kernel<D, IL, PAGED>, grid, fa::kRopeThreads, 0,
                                      s, q, k, v, p, out, dst);
}

template <bool PAGED>
cudaError_t launch_prep_any(const fa::HeadRows& q, const fa::HeadRows& k, const fa::HeadRows& v,
                            const fa::RopeParams& p, const fa::PrepOut& out,
                            const fa::PagedDest& dst, int d, int il, int sms, cudaStream_t s) {
    if (d == 64)
        return il ? launch_prep<64, true, PAGED>(q, k, v, p, out, dst, sms, s)
                  : launch_prep<64, false, PAGED>(q, k, v, p, out, dst, sms, s);
    return il ? launch_prep<128, true, PAGED>(q, k, v, p, out, dst, sms, s)
              : launch_prep<128, false, PAGED>(q, k, v, p, out, dst, sms, s);
}

template <int D, bool IL>
cudaError_t launch_prep_bwd(const fa::HeadRows (&dy)[3], const fa::HeadRows (&x)[2],
                            const fa::HeadRowsOut (&dx)[3], fa::RopeParams p, float* part,
                            float* dwq, float* dwk, int sms, cudaStream_t s) {
    constexpr int TOKENS = fa::kRopeThreads / (D / 8);
    const long long blocks = (static_cast<long long>(p.B) * p.N + TOKENS - 1) / TOKENS;
    const int heads = p.Hq + p.Hkv + (dy[2].p ? p.Hkv : 0);
    const long long units = blocks * heads;
    const int wave = std::min(kMaxBwdCtas / 2, kBwdCtasPerSm * sms);
    long long per_cta = std::max(kMinHeads, (units + wave - 1) / wave);
    if (per_cta >= 2 * kManyHeads) per_cta = (per_cta + 1) / 2;  // still no more than two waves
    const int grid = static_cast<int>((units + per_cta - 1) / per_cta);
    const auto kernel =
        p.wq ? fa::fa_prep_bwd_kernel<D, IL, true> : fa::fa_prep_bwd_kernel<D, IL, false>;
    const cudaError_t e = fa_host::launch_overlapped(
        kernel, dim3(grid), fa::kRopeThreads, 0, s, dy[0], dy[1], dy[2], x[0], x[1], dx[0], dx[1],
        dx[2], p, per_cta, part);
    if (e != cudaSuccess || !p.wq) return e;
    return fa_host::launch_overlapped(fa::fa_dw_reduce_kernel<D>, dim3(2 * D / 8), 1024, 0, s,
                                      static_cast<const float*>(part), grid, dwq, dwk);
}

fa::HeadRows rows_of(const void* p, const long long* s) {
    return {static_cast<const __nv_bfloat16*>(p), s[0], s[1], s[2]};
}
fa::HeadRowsOut rows_out(void* p, const long long* s) {
    return {static_cast<__nv_bfloat16*>(p), s[0], s[1], s[2]};
}

fa_status check_tokens(int B, int N) {
    if (B < 1 || N < 1 || static_cast<long long>(B) * N > (1ll << 30)) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

}  // namespace

extern "C" {

fa_status fa_rope_table(float* table, long long rows, int rope_dim, double base, void* stream) {
    if (!table || rows < 1 || rows > (1ll << 40) || rope_dim < 16 || rope_dim > 128 ||
        rope_dim % 16 || !(std::isfinite(base) && base > 0.0))
        return FA_ERR_INVALID_ARG;
    if (!aligned(table, 16)) return FA_ERR_MISALIGNED;
    int dev, sms;
    unsigned int* err;
    const fa_status st = fa_host::device(&dev, &err, &sms);
    if (st != FA_OK) return st;
    const long long n = rows * (rope_dim / 2);
    const long long grid = std::min<long long>((n + 255) / 256, 8ll * sms);
    fa::fa_rope_table_kernel<<<static_cast<unsigned>(grid), 256, 0,
                               static_cast<cudaStream_t>(stream)>>>(
        reinterpret_cast<float2*>(table), rows, rope_dim / 2, base);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_qk_norm_rope(const void* q, const void* k, const void* v, const long long* strides,
                          const void* q_weight, const void* k_weight, int weight_f32, float eps,
                          const float* rope, long long rope_rows, int rope_dim, int interleaved,
                          const int* positions, void* q_out, void* k_out, void* v_out, int B,
                          int N, int Hq, int Hkv, int d, void* stream) {
    if (!q || !k || !strides || !q_out || !k_out || (v == nullptr) != (v_out == nullptr))
        return FA_ERR_INVALID_ARG;
    if (!q_weight && !rope) return FA_ERR_INVALID_ARG;
    if (interleaved != 0 && interleaved != 1) return FA_ERR_INVALID_ARG;
    fa_status st = check_tokens(B, N);
    if (st == FA_OK) st = check_heads(Hq, Hkv, d);
    if (st == FA_OK)
        st = check_norm_rope(q_weight, k_weight, weight_f32, eps, rope, rope_rows, rope_dim, d);
    if (st != FA_OK) return st;
    // Without positions the tokens have positions 0 .. N - 1.
    if (rope && !positions && rope_rows < N) return FA_ERR_INVALID_ARG;
    if (!strides_ok(strides, v ? 9 : 6)) return FA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
        !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(positions, 4))
        return FA_ERR_MISALIGNED;
    int dev, sms;
    unsigned int* err;
    if ((st = fa_host::device(&dev, &err, &sms)) != FA_OK) return st;
    const fa::RopeParams p = rope_params(q_weight, k_weight, weight_f32, eps, rope, rope_rows,
                                         rope_dim, positions, B, N, Hq, Hkv, err);
    const long long none[3] = {0, 0, 0};
    const fa::PrepOut out = {static_cast<__nv_bfloat16*>(q_out), static_cast<__nv_bfloat16*>(k_out),
                             static_cast<__nv_bfloat16*>(v_out)};
    const cudaError_t e = launch_prep_any<false>(
        rows_of(q, strides), rows_of(k, strides + 3), rows_of(v, v ? strides + 6 : none), p, out,
        fa::PagedDest{}, d, interleaved, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_qk_norm_rope_bwd_workspace_size(int d) {
    return d == 64 || d == 128 ? static_cast<size_t>(kMaxBwdCtas) * 2 * d * sizeof(float) : 0;
}

fa_status fa_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* dv_out,
                              const void* q, const void* k, const long long* strides,
                              const void* q_weight, const void* k_weight, int weight_f32,
                              float eps, const float* rope, long long rope_rows, int rope_dim,
                              int interleaved, const int* positions, void* dq, void* dk, void* dv,
                              const long long* grad_strides, float* dq_weight, float* dk_weight,
                              int B, int N, int Hq, int Hkv, int d, void* workspace,
                              size_t workspace_bytes, void* stream) {
    if (!dq_out || !dk_out || !dq || !dk || !grad_strides ||
        (dv_out == nullptr) != (dv == nullptr))
        return FA_ERR_INVALID_ARG;
    if (!q_weight && !rope) return FA_ERR_INVALID_ARG;
    if (q_weight && (!q || !k || !strides || !dq_weight || !dk_weight)) return FA_ERR_INVALID_ARG;
    if (interleaved != 0 && interleaved != 1) return FA_ERR_INVALID_ARG;
    fa_status st = check_tokens(B, N);
    if (st == FA_OK) st = check_heads(Hq, Hkv, d);
    if (st == FA_OK)
        st = check_norm_rope(q_weight, k_weight, weight_f32, eps, rope, rope_rows, rope_dim, d);
    if (st != FA_OK) return st;
    if (rope && !positions && rope_rows < N) return FA_ERR_INVALID_ARG;
    if (q_weight && !strides_ok(strides, 6)) return FA_ERR_INVALID_ARG;
    if (!strides_ok(grad_strides, dv ? 9 : 6) || !disjoint_rows(grad_strides, B, N, Hq, d) ||
        !disjoint_rows(grad_strides + 3, B, N, Hkv, d) ||
        (dv && !disjoint_rows(grad_strides + 6, B, N, Hkv, d)))
        return FA_ERR_INVALID_ARG;
    if (q_weight && (!workspace || workspace_bytes < fa_qk_norm_rope_bwd_workspace_size(d)))
        return FA_ERR_INVALID_ARG;
    if (!aligned(dq_out, 16) || !aligned(dk_out, 16) || !aligned(dv_out, 16) ||
        (q_weight && (!aligned(q, 16) || !aligned(k, 16))) || !aligned(dq, 16) ||
        !aligned(dk, 16) || !aligned(dv, 16) || !aligned(dq_weight, 4) || !aligned(dk_weight, 4) ||
        !aligned(positions, 4) || !aligned(workspace, 256))
        return FA_ERR_MISALIGNED;
    int dev, sms;
    unsigned int* err;
    if ((st = fa_host::device(&dev, &err, &sms)) != FA_OK) return st;
    const fa::RopeParams p = rope_params(q_weight, k_weight, weight_f32, eps, rope, rope_rows,
                                         rope_dim, positions, B, N, Hq, Hkv, err);
    const long long none[3] = {0, 0, 0};
    const long long hm[3] = {static_cast<long long>(Hq) * N * d, d, static_cast<long long>(N) * d};
    const long long hk[3] = {static_cast<long long>(Hkv) * N * d, d, static_cast<long long>(N) * d};
    const fa::HeadRows dy[3] = {rows_of(dq_out, hm), rows_of(dk_out, hk), rows_of(dv_out, hk)};
    const fa::HeadRows x[2] = {rows_of(q_weight ? q : nullptr, q_weight ? strides : none),
                               rows_of(q_weight ? k : nullptr, q_weight ? strides + 3 : none)};
    const fa::HeadRowsOut dx[3] = {rows_out(dq, grad_strides), rows_out(dk, grad_strides + 3),
                                   rows_out(dv, dv ? grad_strides + 6 : none)};
    float* part = static_cast<float*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const auto launch =
        d == 64 ? (interleaved ? launch_prep_bwd<64, true> : launch_prep_bwd<64, false>)
                : (interleaved ? launch_prep_bwd<128, true> : launch_prep_bwd<128, false>);
    const cudaError_t e = launch(dy, x, dx, p, part, dq_weight, dk_weight, sms, s);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_paged_append(const void* q, const void* k, const void* v, const long long* strides,
                          const void* q_weight, const void* k_weight, int weight_f32, float eps,
                          const float* rope, long long rope_rows, int rope_dim, int interleaved,
                          int pos_offset, const int* seq_start, const int* cache_len,
                          const int* block_table, void* q_out, void* k_pages, void* v_pages,
                          int S, int T, int Hq, int Hkv, int d, int page_size, int num_pages,
                          int max_pages, void* stream) {
    if (!q || !k || !v || !strides || !seq_start || !cache_len || !block_table || !q_out ||
        !k_pages || !v_pages)
        return FA_ERR_INVALID_ARG;
    if (interleaved != 0 && interleaved != 1) return FA_ERR_INVALID_ARG;
    if (S < 1 || T < 0 || T > (1 << 30) || num_pages < 1 || max_pages < 1 || pos_offset < 0)
        return FA_ERR_INVALID_ARG;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
        return FA_ERR_INVALID_ARG;
    fa_status st = check_heads(Hq, Hkv, d);
    if (st == FA_OK)
        st = check_norm_rope(q_weight, k_weight, weight_f32, eps, rope, rope_rows, rope_dim, d);
    if (st != FA_OK) return st;
    if (!strides_ok(strides, 6)) return FA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
        !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(seq_start, 4) ||
        !aligned(cache_len, 4) || !aligned(block_table, 4))
        return FA_ERR_MISALIGNED;
    if (T == 0) return FA_OK;
    int dev, sms;
    unsigned int* err;
    if ((st = fa_host::device(&dev, &err, &sms)) != FA_OK) return st;
    const fa::RopeParams p = rope_params(q_weight, k_weight, weight_f32, eps, rope, rope_rows,
                                         rope_dim, nullptr, 1, T, Hq, Hkv, err);
    fa::PagedDest dst;
    dst.seq_start = seq_start;
    dst.cache_len = cache_len;
    dst.block_table = block_table;
    dst.S = S;
    dst.max_pages = max_pages;
    dst.page_shift = 0;
    while ((1 << dst.page_shift) < page_size) ++dst.page_shift;
    dst.num_pages = num_pages;
    dst.pos_offset = pos_offset;
    dst.q_out = static_cast<__nv_bfloat16*>(q_out);
    dst.k_pages = static_cast<__nv_bfloat16*>(k_pages);
    dst.v_pages = static_cast<__nv_bfloat16*>(v_pages);
    const long long sq[3] = {0, strides[0], strides[1]}, sk[3] = {0, strides[2], strides[3]},
                    sv[3] = {0, strides[4], strides[5]};
    const cudaError_t e =
        launch_prep_any<true>(rows_of(q, sq), rows_of(k, sk), rows_of(v, sv), p, fa::PrepOut{},
                              dst, d, interleaved, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
