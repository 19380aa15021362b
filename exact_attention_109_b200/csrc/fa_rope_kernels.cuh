// fa_rope_kernels.cuh -- what stands between a projection and attention: the
// RMS norm of every head's query and key row, the position rotation, and the
// move from the projection's token-major rows into the layout the attention
// kernels read ([B, H, N, d], or the pages of a cache), in one pass.
//
// Forward, per row x of d values:  rstd = (mean(x^2) + eps)^(-1/2),
// u = x * rstd * w, and every pair (a, b) of u's first rope_dim values turned
// by its angle: (a cos - b sin, b cos + a sin).  The pairs are (i, i + rope/2)
// or, interleaved, (2i, 2i + 1).
// Backward, with g the upstream gradient turned back by the same angles:
//   dw = sum over rows of g * x * rstd
//   dx = rstd * (g w - x rstd * mean(g w x rstd)).
//
// These passes are bound by HBM: 2 bytes read and 2 written per value against
// about ten fp32 operations.  So a row is held in registers by d / 8 lanes
// (one 16-byte access each; 16 rows of 128 or 32 of 64 per CTA), its sums go
// through shuffles, and everything that depends on the token alone (sequence,
// page, angles) is read once and used for all heads the CTA walks.  Rows come
// in through a ring of shared memory that each thread fills and reads for
// itself.  All arithmetic is fp32, rounded once on the way out.
//
// Measured, 16384 tokens of 16 query, 16 key and 16 value heads of 128: forward
// 67.5 us for 407 MB (92 % of the measured copy bandwidth; 87 us with the rows
// in flight held in registers), backward 97 us for 541 MB (85 %; 191 us so).
// The same reads and writes without the arithmetic take the backward 93 us.
// Packed fp32 pairs and a loader without branches took 4 and 9 % off.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sm100_ptx.cuh"

namespace fa {

// Rows of one tensor: element strides of the batch (or nothing, for packed
// tokens), the token and the head; the d values of a row are contiguous.
struct HeadRows {
    const __nv_bfloat16* p;
    long long sb, sn, sh;
};
struct HeadRowsOut {
    __nv_bfloat16* p;
    long long sb, sn, sh;
};

struct RopeParams {
    const float2* table;   // [rows][rope_dim / 2] (cos, sin), or null
    long long rows;
    int rope_dim;          // a multiple of 16; 0 without a table
    const int* positions;  // [B][N], or null: token n has position n
    const void* wq;        // [d], or null: no norm
    const void* wk;
    int w_f32;             // the weights are fp32 (else bf16)
    float eps;
    int B, N, Hq, Hkv;
    int heads_per_cta;
    unsigned int* err;
};

// Where a paged cache takes the tokens (PAGED).
struct PagedDest {
    const int* seq_start;    // [S + 1]
    const int* cache_len;    // [S]
    const int* block_table;  // [S][max_pages]
    int S, max_pages, page_shift, num_pages, pos_offset;
    __nv_bfloat16* q_out;    // [T][Hq][d]
    __nv_bfloat16* k_pages;  // [num_pages][Hkv][page][d]
    __nv_bfloat16* v_pages;
};

struct PrepOut {
    __nv_bfloat16 *q, *k, *v;  // [B][H][N][d]; v may be null
};

constexpr int kRopeThreads = 256;

// The eight bf16 of a lane's 16 bytes as four pairs of fp32 (for packed
// arithmetic), and back.
__device__ __forceinline__ void widen8(const uint4& w, uint64_t (&x)[4]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = f2_pack(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}

__device__ __forceinline__ uint4 narrow8(const uint64_t (&x)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        f2_unpack(x[i], lo, hi);
        u[i] = pack_bf16x2(lo, hi);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ float sum_pair(uint64_t x) {
    float lo, hi;
    f2_unpack(x, lo, hi);
    return lo + hi;
}

__device__ __forceinline__ float weight_at(const void* w, int f32, int i) {
    return f32 ? static_cast<const float*>(w)[i]
               : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}

// Sum over the LANES (8 or 16) lanes that share a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The same of two numbers: lanes of one parity add the first, the others the
// second, and the parities exchange them (five shuffles instead of eight).
template <int LANES>
__device__ __forceinline__ void row_sum2(float& a, float& b, int lane) {
    const bool odd = lane & 1;
    float keep = odd ? b : a;
    keep += __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
#pragma unroll
    for (int o = 2; o < LANES; o <<= 1) keep += __shfl_xor_sync(0xffffffffu, keep, o);
    const float other = __shfl_xor_sync(0xffffffffu, keep, 1);
    a = odd ? other : keep;
    b = odd ? keep : other;
}

// One lane's share of the rotation: it holds values [8c, 8c + 8) of a row.
// Values beyond rope_dim take cosine 1, sine 0 and a partner of 0.
template <int D, bool INTERLEAVED>
struct Turn {
    static constexpr int LANES = D / 8;
    int src;        // lane that holds the other members of the pairs
    int other;      // index of the pair partner of value 8c (INTERLEAVED: unused)
    uint32_t seen;  // mask of the partners' bits
    uint64_t c[4];  // cosines, and sines with the sign that a value's partner takes
    uint64_t s[4];  // in the turn (minus for a pair's first member)

    // c and s of every value, from the token's row of the table.
    __device__ __forceinline__ void load(const RopeParams& p, long long pos, int lane) {
        const int col = lane & (LANES - 1), e0 = 8 * col;
        src = lane;
        other = e0;
        seen = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = f2_pack(1.f, 1.f);
            s[i] = 0ull;
        }
        if (e0 >= p.rope_dim) return;
        seen = 0xffffffffu;
        const float4* row =
            reinterpret_cast<const float4*>(p.table + pos * (p.rope_dim / 2));
        if constexpr (INTERLEAVED) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // two pairs per 16 bytes
                const float4 f = __ldg(row + 2 * col + i);
                c[2 * i] = f2_pack(f.x, f.x);
                s[2 * i] = f2_pack(-f.y, f.y);
                c[2 * i + 1] = f2_pack(f.z, f.z);
                s[2 * i + 1] = f2_pack(-f.w, f.w);
            }
        } else {
            const int half = p.rope_dim / 2;
            const bool second = e0 >= half;
            const float sign = second ? 1.f : -1.f;
            other = second ? e0 - half : e0 + half;
            src = (lane & ~(LANES - 1)) | (other >> 3);
            const int i0 = second ? e0 - half : e0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = __ldg(row + i0 / 2 + i);
                c[i] = f2_pack(f.x, f.z);
                s[i] = f2_pack(sign * f.y, sign * f.w);
            }
        }
    }

    __device__ __forceinline__ int partner_index(int e0, int j) const {
        return INTERLEAVED ? (e0 + (j ^ 1)) : (other + j);
    }
    // The pair partners of the eight values in `w` (all lanes take part).
    __device__ __forceinline__ void partners(const uint4& w, uint64_t (&y)[4]) const {
        uint4 t;
        if constexpr (INTERLEAVED) {
            t = make_uint4(__byte_perm(w.x, 0, 0x1032), __byte_perm(w.y, 0, 0x1032),
                           __byte_perm(w.z, 0, 0x1032), __byte_perm(w.w, 0, 0x1032));
        } else {
            t.x = __shfl_sync(0xffffffffu, w.x, src);
            t.y = __shfl_sync(0xffffffffu, w.y, src);
            t.z = __shfl_sync(0xffffffffu, w.z, src);
            t.w = __shfl_sync(0xffffffffu, w.w, src);
        }
        widen8(make_uint4(t.x & seen, t.y & seen, t.z & seen, t.w & seen), y);
    }
};

// The position of a token, checked against the table; a bad one is reported
// and read as 0.
__device__ __forceinline__ long long checked_position(const RopeParams& p, long long pos,
                                                      bool active) {
    if (!p.table) return 0;
    if (pos >= 0 && pos < p.rows) return pos;
    if (active) atomicOr(p.err, kErrIndex);
    return 0;
}

// The sequence of packed token t: the last s with seq_start[s] <= t.  One
// token per sequence is a decoding server's usual call, so s = t is tried
// before the binary search.  The caller has checked that t lies below
// seq_start[S].
__device__ __forceinline__ int sequence_of(const int* seq_start, int S, int t) {
    if (t < S && seq_start[t] <= t && t < seq_start[t + 1]) return t;
    int lo = 0, hi = S - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (seq_start[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Each thread's rows on their way in: SLOTS slots of two 16-byte pieces that
// it alone writes (with asynchronous copies) and reads, so no barrier is
// needed and the bytes in flight do not cost registers.
template <int SLOTS>
struct RowRing {
    uint32_t base;  // of this thread's piece 0 in slot 0
    static constexpr uint32_t PIECE = kRopeThreads * 16u, SLOT = 2u * PIECE;
    static constexpr int BYTES = SLOTS * static_cast<int>(SLOT);

    __device__ __forceinline__ void put(int slot, int piece, const __nv_bfloat16* src) const {
        cp_async16(base + slot * SLOT + piece * PIECE, src);
    }
    static __device__ __forceinline__ void commit() {
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // All groups but the newest SLOTS - 2 have landed: with SLOTS - 1 of them
    // committed ahead of the step that reads, that step's.
    static __device__ __forceinline__ void wait() {
        asm volatile("cp.async.wait_group %0;" ::"n"(SLOTS - 2) : "memory");
    }
    __device__ __forceinline__ uint4 get(int slot, int piece) const {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(base + slot * SLOT + piece * PIECE)
                     : "memory");
        return v;
    }
    static __device__ __forceinline__ int next(int slot) {
        return slot + 1 == SLOTS ? 0 : slot + 1;
    }
};

// The heads [a, z) of part 0, 1, 2 (queries, keys, values) among [h0, h1).
struct PartRange {
    int first, count, a, z;
    __device__ __forceinline__ PartRange(const RopeParams& p, int part, int h0, int h1)
        : first(part == 0 ? 0 : p.Hq + (part - 1) * p.Hkv),
          count(part == 0 ? p.Hq : p.Hkv),
          a(max(h0, first)),
          z(min(h1, first + count)) {}
};

// Grid: x over blocks of 256 / (D / 8) tokens, y over groups of heads.  The
// heads are the Hq query heads, then Hkv key heads, then (with v) Hkv value
// heads, which are moved unchanged.
template <int D, bool INTERLEAVED, bool PAGED>
__global__ void __launch_bounds__(kRopeThreads, 3)
    fa_prep_kernel(const HeadRows q, const HeadRows k, const HeadRows v, const RopeParams p,
                   const PrepOut out, const PagedDest dst) {
    constexpr int LANES = D / 8, TOKENS = kRopeThreads / LANES, SLOTS = 4;
    __shared__ __align__(16) uint8_t ring_mem[RowRing<SLOTS>::BYTES];
    const RowRing<SLOTS> ring{smem_u32(ring_mem) + threadIdx.x * 16u};
    const int lane = threadIdx.x & 31;
    const int col = threadIdx.x & (LANES - 1), e0 = 8 * col;
    const long long total = static_cast<long long>(p.B) * p.N;
    long long row = static_cast<long long>(blockIdx.x) * TOKENS + threadIdx.x / LANES;
    bool active = row < total;
    if (!active) row = total - 1;
    const long long b = PAGED ? 0 : row / p.N;
    const long long n = PAGED ? row : row - b * p.N;
    const int heads = p.Hq + p.Hkv + (v.p ? p.Hkv : 0);
    const int h0 = blockIdx.y * p.heads_per_cta;
    const int h1 = min(h0 + p.heads_per_cta, heads);

    // The loader runs SLOTS - 1 steps ahead; a step is two heads of one part.
    int load_part = -1, load_left = 0, load_slot = 0;
    const __nv_bfloat16* load_src = nullptr;
    long long load_step = 0;
    auto load = [&]() {
        while (load_left == 0 && load_part < 2) {
            const PartRange r(p, ++load_part, h0, h1);
            if (r.a >= r.z) continue;
            const HeadRows& in = load_part == 0 ? q : load_part == 1 ? k : v;
            load_left = r.z - r.a;
            load_src = in.p + b * in.sb + n * in.sn + (r.a - r.first) * in.sh + e0;
            load_step = in.sh;
        }
        if (load_left > 0) {
            ring.put(load_slot, 0, load_src);
            if (load_left > 1) ring.put(load_slot, 1, load_src + load_step);
            load_src += 2 * load_step;
            load_left = max(0, load_left - 2);
            load_slot = ring.next(load_slot);
        }
        ring.commit();
    };
    grid_dependency_wait();
    grid_launch_dependents();
#pragma unroll
    for (int i = 0; i < SLOTS - 1; ++i) load();

    long long pos;
    long long page_row = -1;  // row of the token in its page, over all pages; -1: nowhere
    long long page = 0;
    if constexpr (PAGED) {
        const int t = static_cast<int>(row);
        if (t >= dst.seq_start[dst.S] || t < dst.seq_start[0]) active = false;  // no sequence's
        pos = 0;
        if (active) {
            const int s = sequence_of(dst.seq_start, dst.S, t);
            const int have = dst.cache_len[s];
            // In 64 bits: a start far below 0, which is reported below, must not
            // turn the key's index, and with it the table's, negative.
            const long long at = static_cast<long long>(have) + t - dst.seq_start[s];
            const long long slot = at >> dst.page_shift;
            pos = at + dst.pos_offset;
            if (have >= 0 && slot < dst.max_pages) {
                page = dst.block_table[static_cast<long long>(s) * dst.max_pages + slot];
                if (page >= 0 && page < dst.num_pages) page_row = at - (slot << dst.page_shift);
            }
            if (page_row < 0) atomicOr(p.err, kErrIndex);
        }
        if (blockIdx.x + blockIdx.y == 0)
            for (int i = threadIdx.x; i < dst.S; i += kRopeThreads) {
                const int a = dst.seq_start[i], z = dst.seq_start[i + 1];
                if (a < 0 || z < a || z > p.N) atomicOr(p.err, kErrIndex);
            }
    } else {
        pos = p.positions ? p.positions[row] : n;
    }
    pos = checked_position(p, pos, active);
    const bool norm = p.wq != nullptr;

    int slot = 0;
#pragma unroll 1
    for (int part = 0; part < 3; ++part) {
        const PartRange r(p, part, h0, h1);
        if (r.a >= r.z) continue;
        // Destination of the first head and the step to the next.
        __nv_bfloat16* to;
        long long step;
        bool write = active;
        if constexpr (PAGED) {
            if (part == 0) {
                to = dst.q_out + (row * p.Hq + r.a) * D + e0;
                step = D;
            } else {
                write = page_row >= 0;
                step = static_cast<long long>(D) << dst.page_shift;
                to = (part == 1 ? dst.k_pages : dst.v_pages) +
                     (page * p.Hkv + (r.a - r.first)) * step + (write ? page_row : 0) * D + e0;
            }
        } else {
            step = static_cast<long long>(p.N) * D;
            to = (part == 0 ? out.q : part == 1 ? out.k : out.v) +
                 (b * r.count + (r.a - r.first)) * step + n * D + e0;
        }
        if (part == 2) {
#pragma unroll 1
            for (int h = r.a; h < r.z; h += 2) {
                ring.wait();
                const uint4 w0 = ring.get(slot, 0), w1 = ring.get(slot, 1);
                slot = ring.next(slot);
                load();
                if (write) *reinterpret_cast<uint4*>(to) = w0;
                if (write && h + 1 < r.z) *reinterpret_cast<uint4*>(to + step) = w1;
                to += 2 * step;
            }
            continue;
        }
        // y_j = rstd * (x_j * own_j + partner_j * cross_j)
        Turn<D, INTERLEAVED> turn;
        turn.load(p, pos, lane);
        uint64_t own[4], cross[4];
        const void* wt = part == 0 ? p.wq : p.wk;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            own[i] = turn.c[i];
            cross[i] = turn.s[i];
            if (norm) {
                const int o = turn.partner_index(e0, 2 * i), o1 = turn.partner_index(e0, 2 * i + 1);
                own[i] = fmul2(own[i], f2_pack(weight_at(wt, p.w_f32, e0 + 2 * i),
                                               weight_at(wt, p.w_f32, e0 + 2 * i + 1)));
                cross[i] = fmul2(cross[i], f2_pack(weight_at(wt, p.w_f32, o),
                                                   weight_at(wt, p.w_f32, o1)));
            }
        }
#pragma unroll 1
        for (int h = r.a; h < r.z; h += 2) {
            ring.wait();
            uint4 w[2];
            w[0] = ring.get(slot, 0);
            w[1] = h + 1 < r.z ? ring.get(slot, 1) : make_uint4(0u, 0u, 0u, 0u);
            slot = ring.next(slot);
            load();
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint64_t x[4], xp[4], y[4];
                widen8(w[u], x);
                turn.partners(w[u], xp);
                float rstd = 1.f;
                if (norm) {
                    uint64_t ss = fmul2(x[0], x[0]);
#pragma unroll
                    for (int i = 1; i < 4; ++i) ss = ffma2(x[i], x[i], ss);
                    rstd = rsqrtf(row_sum<LANES>(sum_pair(ss)) * (1.f / D) + p.eps);
                }
                const uint64_t rstd2 = f2_pack(rstd, rstd);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[i] = fmul2(rstd2, ffma2(xp[i], cross[i], fmul2(x[i], own[i])));
                if (h + u < r.z && write) *reinterpret_cast<uint4*>(to + u * step) = narrow8(y);
            }
            to += 2 * step;
        }
    }
}

// Gradients of fa_prep_kernel's training form.  The heads of all token blocks
// are numbered block by block, and CTA c takes numbers [c, c + 1) * per_cta: a
// few whole blocks and two parts of one.  With a norm it leaves its sums of dw
// for queries and keys in `part` [CTAs][2][D], which fa_dw_reduce_kernel adds
// up in a fixed order.
template <int D, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, 2)
    fa_prep_bwd_kernel(const HeadRows dyq, const HeadRows dyk, const HeadRows dyv,
                       const HeadRows xq, const HeadRows xk, const HeadRowsOut dq,
                       const HeadRowsOut dk, const HeadRowsOut dv, const RopeParams p,
                       long long per_cta, float* part_dw) {
    constexpr int LANES = D / 8, TOKENS = kRopeThreads / LANES, SLOTS = 6;
    using Ring = RowRing<SLOTS>;
    __shared__ __align__(16) uint8_t ring_mem[Ring::BYTES];
    const Ring ring{smem_u32(ring_mem) + threadIdx.x * 16u};
    const int lane = threadIdx.x & 31;
    const int col = threadIdx.x & (LANES - 1), e0 = 8 * col;
    const long long total = static_cast<long long>(p.B) * p.N;
    const int heads = p.Hq + p.Hkv + (dyv.p ? p.Hkv : 0);
    const long long first_head = blockIdx.x * per_cta;
    const long long last_head =
        min(first_head + per_cta, (total + TOKENS - 1) / TOKENS * heads);
    uint64_t dw[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[0][i] = dw[1][i] = 0ull;

    // An item: the token (b, n) and its heads [h0, h1).
    struct Item {
        long long row, b, n;
        bool active;
        int h0, h1;
    };
    auto item_at = [&](long long at) {
        Item x;
        const long long tb = at / heads;
        x.h0 = static_cast<int>(at - tb * heads);
        x.h1 = static_cast<int>(min(static_cast<long long>(heads), x.h0 + (last_head - at)));
        x.row = tb * TOKENS + threadIdx.x / LANES;
        x.active = x.row < total;
        if (!x.active) x.row = total - 1;
        x.b = x.row / p.N;
        x.n = x.row - x.b * p.N;
        return x;
    };
    // The loader runs SLOTS - 1 steps ahead, over the borders of items.  A
    // step is a head's gradient and (NORM) row, or two value heads (one, twice,
    // where their number is odd).
    long long load_at = first_head;
    int load_part = -1, load_left = 0;
    const __nv_bfloat16 *load_a = nullptr, *load_b = nullptr;
    long long step_a = 0, step_b = 0;
    auto seek = [&]() {
        while (load_left == 0 && load_at < last_head) {
            const Item x = item_at(load_at);
            if (++load_part == 3) {
                load_part = -1;
                load_at += x.h1 - x.h0;
                continue;
            }
            const PartRange r(p, load_part, x.h0, x.h1);
            if (r.a >= r.z) continue;
            const HeadRows& dy = load_part == 0 ? dyq : load_part == 1 ? dyk : dyv;
            load_left = r.z - r.a;
            load_a = dy.p + x.b * dy.sb + x.n * dy.sn + (r.a - r.first) * dy.sh + e0;
            load_b = load_a;
            step_a = step_b = dy.sh;
            if (load_part == 2) {
                if (load_left % 2 == 0) {
                    load_b = load_a + dy.sh;
                    step_a = step_b = 2 * dy.sh;
                    load_left /= 2;
                }
            } else if (NORM) {
                const HeadRows& in = load_part == 0 ? xq : xk;
                load_b = in.p + x.b * in.sb + x.n * in.sn + (r.a - r.first) * in.sh + e0;
                step_b = in.sh;
            }
        }
    };
    auto load = [&](int slot) {
        if (load_left > 0) {
            ring.put(slot, 0, load_a);
            if (NORM || load_part == 2) ring.put(slot, 1, load_b);
            load_a += step_a;
            load_b += step_b;
            if (--load_left == 0) seek();
        }
        ring.commit();
    };
    grid_dependency_wait();
    grid_launch_dependents();
    seek();
#pragma unroll
    for (int i = 0; i < SLOTS - 1; ++i) load(i);

    // The slot that the last step read is free again.
    int slot = 0, freed = SLOTS - 1;
    auto take = [&](uint4& a, uint4& b) {
        ring.wait();
        a = ring.get(slot, 0);
        b = ring.get(slot, 1);
        load(freed);
        freed = slot;
        slot = ring.next(slot);
    };
#pragma unroll 1
    for (long long at = first_head; at < last_head;) {
        const Item x = item_at(at);
        at += x.h1 - x.h0;
        Turn<D, INTERLEAVED> turn;
        turn.load(p, checked_position(p, p.positions ? p.positions[x.row] : x.n, x.active), lane);

#pragma unroll
        for (int part = 0; part < 3; ++part) {
            const PartRange r(p, part, x.h0, x.h1);
            if (r.a >= r.z) continue;
            const HeadRowsOut& dx = part == 0 ? dq : part == 1 ? dk : dv;
            __nv_bfloat16* to = dx.p + x.b * dx.sb + x.n * dx.sn + (r.a - r.first) * dx.sh + e0;
            if (part == 2) {
                const bool two = (r.z - r.a) % 2 == 0;
#pragma unroll 1
                for (int h = r.a; h < r.z; h += two ? 2 : 1) {
                    uint4 w0, w1;
                    take(w0, w1);
                    if (x.active) *reinterpret_cast<uint4*>(to) = w0;
                    if (x.active && two) *reinterpret_cast<uint4*>(to + dx.sh) = w1;
                    to += two ? 2 * dx.sh : dx.sh;
                }
                continue;
            }
            uint64_t w[4];
            if constexpr (NORM) {
                const void* wt = part == 0 ? p.wq : p.wk;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = f2_pack(weight_at(wt, p.w_f32, e0 + 2 * i),
                                   weight_at(wt, p.w_f32, e0 + 2 * i + 1));
            }
#pragma unroll 1
            for (int h = r.a; h < r.z; ++h) {
                uint4 gr, xr;
                take(gr, xr);
                uint64_t g[4], gp[4], y[4];
                widen8(gr, g);
                turn.partners(gr, gp);
#pragma unroll
                for (int i = 0; i < 4; ++i)  // the turn's transpose: g c - gp s
                    y[i] = fsub2(fmul2(g[i], turn.c[i]), fmul2(gp[i], turn.s[i]));
                if constexpr (NORM) {
                    uint64_t v[4], t[4], ss2, gx2;
                    widen8(xr, v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        t[i] = fmul2(y[i], w[i]);
                        ss2 = i ? ffma2(v[i], v[i], ss2) : fmul2(v[i], v[i]);
                        gx2 = i ? ffma2(t[i], v[i], gx2) : fmul2(t[i], v[i]);
                    }
                    float ss = sum_pair(ss2), gx = sum_pair(gx2);
                    row_sum2<LANES>(ss, gx, lane);
                    const float rstd = rsqrtf(ss * (1.f / D) + p.eps);
                    const float along = gx * rstd * (-1.f / D) * rstd;
                    const uint64_t rstd2 = f2_pack(rstd, rstd), along2 = f2_pack(along, along);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint64_t xh = fmul2(v[i], rstd2);
                        if (x.active) dw[part][i] = ffma2(y[i], xh, dw[part][i]);
                        y[i] = ffma2(xh, along2, fmul2(t[i], rstd2));
                    }
                }
                if (x.active) *reinterpret_cast<uint4*>(to) = narrow8(y);
                to += dx.sh;
            }
        }
    }
    if constexpr (!NORM) return;

    // The CTA's sums: over the rows of each warp by shuffles, then over the
    // warps through shared memory (the ring's: its copies have all been read).
    auto red = reinterpret_cast<float(*)[2][D]>(ring_mem);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float lo, hi;
            f2_unpack(dw[i][j / 2], lo, hi);
            float x = j & 1 ? hi : lo;
#pragma unroll
            for (int o = LANES; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (lane < LANES) red[threadIdx.x >> 5][i][e0 + j] = x;
        }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * D; c += kRopeThreads) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kRopeThreads / 32; ++w) x += red[w][c / D][c % D];
        part_dw[static_cast<long long>(blockIdx.x) * 2 * D + c] = x;
    }
}

// dw[c] = sum over `ctas` of part[cta][c]: 8 columns per CTA, 128 rows of
// threads, always in the same order.
template <int D>
__global__ void __launch_bounds__(1024)
    fa_dw_reduce_kernel(const float* part, int ctas, float* dwq, float* dwk) {
    __shared__ float red[32][9];
    const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
    const int c = blockIdx.x * 8 + x;
    grid_dependency_wait();
    float s = 0.f;
#pragma unroll 5
    for (int r = y; r < ctas; r += 128) s += part[static_cast<long long>(r) * 2 * D + c];
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    if ((threadIdx.x & 31) < 8) red[threadIdx.x >> 5][x] = s;
    __syncthreads();
    if (threadIdx.x >= 256) return;
    s = red[threadIdx.x & 31][threadIdx.x >> 5];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) {
        const int col = blockIdx.x * 8 + (threadIdx.x >> 5);
        (col < D ? dwq : dwk)[col % D] = s;
    }
}

// table[r][i] = (cos, sin) of r * base^(-2i / rope_dim), from 64-bit angles:
// a position of 10^6 times a 32-bit frequency would be off by 0.06 rad.
__global__ void fa_rope_table_kernel(float2* table, long long rows, int half, double base) {
    const long long n = rows * half;
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<long long>(gridDim.x) * blockDim.x) {
        const long long r = i / half;
        const double angle = static_cast<double>(r) *
                             pow(base, -static_cast<double>(i - r * half) / half);
        double s, c;
        sincos(angle, &s, &c);
        table[i] = make_float2(static_cast<float>(c), static_cast<float>(s));
    }
}

}  // namespace fa
