// fa_paged_kernels.cuh -- attention of a batch's new tokens over a paged
// key/value cache, behind a prefix that all sequences share.
//
// The keys a token sees are the shared prefix and its own sequence's rows.
// Softmax over a union of key sets is the log-sum-exp merge of the parts
// (iplexlaw blog, "Tiling preserves the attention calculation"), so each part
// is computed where it is cheap and the parts are merged:
//
//  * Prefix (fa_prefix_kernel).  All T tokens of the batch see the same keys,
//    so the T * G query rows of a key head (G query heads per key head) form
//    one dense matrix against it: every key and value is read once for 128 or
//    256 rows instead of once per sequence.  That is a matrix product for the
//    tensor cores: tcgen05.mma with 128-row tiles, accumulators in TMEM, K and
//    V pages brought in by TMA.  The prefix is cut into splits so that every
//    SM streams.
//  * Own rows (fa_own_kernel).  One sequence's keys serve only its own n * G
//    rows (a handful), so this part is bound by reading the cache; a 128-row
//    tile would be mostly padding.  Warps use 8- or 16-row mma.sync tiles on keys
//    streamed through shared memory by TMA.  The key blocks of all sequences
//    and heads form one line that is cut into equal pieces, one per CTA, so
//    ragged lengths leave no SM idle and the loads never stop between them.
//    A prefix that 16 rows or fewer read is one more sequence of this line: one
//    tile of it, or two of 8 rows behind a prefix that L2 holds.
//  * fa_paged_merge_kernel joins the partial results of a row.
//
// A page is [page rows][d] per head, contiguous, so one TMA box of
// min(page, 64) rows x 64 columns lies within a page; a key block is filled by
// as many boxes as its rows span.  Boxes that start behind the last key are
// not loaded.  Rows behind the last key within a loaded box, and whatever the
// buffer held where no box was loaded, may be anything (NaN included): their
// scores are replaced by -inf, and their V rows by zeros, because a weight of
// zero times NaN is NaN.
#pragma once

#include "sm100_ptx.cuh"

namespace fa {

struct PagedParams {
    const __nv_bfloat16* q;   // [T][Hq][D]
    const int* block_table;   // [S][max_pages]
    const int* seq_start;     // [S + 1]
    const int* kv_len;        // [S]
    const int* prefix_pages;  // [ceil(prefix_len / page)]
    const __nv_bfloat16* v_pages;  // [num_pages][Hkv][page][D], for not_finite_values
    __nv_bfloat16* o;         // [T][Hq][D]
    float* lse;               // [T][Hq], natural log
    // Partial results, normalised, with their log-sum-exp (base 2; -inf:
    // nothing seen, O not written).  Row (x * Hkv + head) * R + i holds query
    // row i of slot x: the prefix's splits, then (with a prefix) the sequences'
    // own keys where one CTA had them all.  Behind the slots, row
    // piece_row + (2 c + w) * 16 + i holds row i of a tile that CTA c of the
    // line had a part of: its first tile (w = 0) or its last.
    float* part_o;
    float* part_lse;
    long long piece_row;
    // [2][Hkv][R] (own keys; prefix in the line): how many CTAs had a part of
    // the row's tile, and (2 c + w) * 16 + i of the first.
    int2* pieces;
    unsigned int* err;
    int S, T, Hq, Hkv, G, R;  // R = T * G query rows per key head
    int page_shift, box_shift;  // log2 of the page's and of a TMA box's rows
    int num_pages, max_pages, max_new;
    int prefix_len, prefix_splits, prefix_chunk, row_tiles;
    int prefix_slots;         // partial results of the prefix: splits, or twice that (HALVES)
    int prefix_in_line;       // the prefix is one more sequence of the line
    int slots, line_ctas;
    int tile_rows;            // query rows of a tile of the line, 8 or 16
    float scale_log2;         // scale * log2(e)
};

// Key blocks that a CTA of the line takes at least, and what a tile costs
// beside its keys, in blocks: reading Q, joining the warps, writing.
constexpr int kLineMinBlocks = 2;
constexpr int kLineTileBlocks = 2;
constexpr int kPieceRows = 16;  // rows of a CTA's part of a tile, in the workspace

// Plane of (page, head) in the page tensors' maps.  A page out of range is
// reported and mapped behind the tensor, where TMA fills with zeros.
__device__ __forceinline__ int page_plane(const PagedParams& p, int page, int head) {
    if (page >= 0 && page < p.num_pages) return page * p.Hkv + head;
    atomicOr(p.err, kErrIndex);
    return p.num_pages * p.Hkv;
}

// ------------------------------------------------------------------ prefix

template <int D, int TILES>
struct PrefixTraits {
    static_assert(D == 64 || D == 128, "head dim");
    static_assert(TILES == 1 || TILES == 2, "query tiles per CTA");
    static constexpr int BN = 128;
    static constexpr int CHUNKS = D / 64;
    static constexpr int CHUNK_BYTES = 128 * 128;
    static constexpr int TILE_BYTES = 128 * D * 2;
    // K and V blocks of 128 rows; as many as fit beside the query tiles.
    static constexpr int NSLOT = D == 128 ? (TILES == 2 ? 4 : 6) : 10;
    static constexpr int Q_OFF = 0;
    static constexpr int KV_OFF = Q_OFF + TILES * TILE_BYTES;
    static constexpr int BAR_OFF = KV_OFF + NSLOT * TILE_BYTES;
    // q, full[NSLOT], empty[NSLOT], s_full[2], p_ready[2], o_final[2], o_done,
    // v_last, v_fixed, mma_done
    static constexpr int NBAR = 1 + 2 * NSLOT + 6 + 4;
    static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
    static constexpr int SMEM_BYTES = MISC_OFF + 16 + 1024;  // + alignment slack
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
    static constexpr int NUM_THREADS = 128 * (TILES + 1);
    static constexpr int MMA_WARP = 4 * TILES;
    static constexpr int LOAD_WARP = MMA_WARP + 1;
    static constexpr int FIX_WARP = MMA_WARP + 2;
    // Register split with two tiles (384 threads leave 168 each): the softmax
    // holds a whole block of scores.
    static constexpr uint32_t REG_SOFTMAX = 208;
    static constexpr uint32_t REG_CONTROL = 88;
    static constexpr int REG_BUDGET =
        TILES == 2 ? 128 * (2 * static_cast<int>(REG_SOFTMAX) + static_cast<int>(REG_CONTROL)) : 0;
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t IDESC_S = idesc_bf16_f32(128, BN, 0, 0);
    static constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, 0, 1);
    static constexpr float TAU = 8.0f;  // deferred-rescale threshold (log2 units)
};

// Keys [key, kend) of the prefix, heads of 64: the sums of their values that are
// not finite, of columns 2 * lane and 2 * lane + 1 (0 where all are).
__device__ __noinline__ float2 not_finite_values(const __nv_bfloat16* v_pages, const int* pages,
                                                 int num_pages, int Hkv, int head, int page_shift,
                                                 int key, int kend) {
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll 4
    for (; key < kend; ++key) {
        const int page = pages[key >> page_shift];
        if (page < 0 || page >= num_pages) continue;  // reported by the loading warp
        const long long row = ((static_cast<long long>(page) * Hkv + head) << page_shift) +
                              (key & ((1 << page_shift) - 1));
        const uint32_t w =
            *reinterpret_cast<const uint32_t*>(v_pages + row * 64 + 2 * (threadIdx.x & 31));
        if ((w & 0x7f80u) == 0x7f80u) sum.x += __uint_as_float(w << 16);
        if ((w & 0x7f800000u) == 0x7f800000u) sum.y += __uint_as_float(w & 0xffff0000u);
    }
    return sum;
}

// One CTA: 128 * TILES query rows of a key head against one split of the
// prefix.  Roles as in fa_fwd_kernel: a softmax warpgroup per query tile (one
// thread per row), a thread that issues the MMAs, a warp that loads; one more
// warp zeroes the value rows behind the last key.  With one tile the scores
// have two TMEM buffers, so that the tensor core computes the next block's
// while the softmax works on this one's; with two tiles each has its own and
// they alternate.  TMEM columns: scores / P at 0 and 128, O at 256 (+ D).
//
// Measured with two tiles and heads of 128: 1.83 us a block of 128 keys for 256
// rows, 1.36 PFLOP/s over 144 CTAs (84 % of the measured bf16 peak), bound by a
// tile's chain of score product, softmax and value product; set-up 4 us, the
// partial results 3 us.  1024 rows behind 65536 keys of 4 heads: 113 to 125 us.
// One tile, heads of 64: 1.05 us a block, the softmax of the warps that have
// rows, 0.9 with HALVES.  Moving exponentials to the FMA pipes or handing P over in halves
// changed nothing or made it slower.
//
// HALVES: at most 64 query rows.  They stand in the tile twice, and the two
// copies take a half of every block's keys each, so that all four softmax warps
// have work and half as much of it; the copies' results are joined like those
// of two splits.  The value product runs over all keys for both, with weights of
// zero for the other copy's, and zero times an infinity is NaN: where an output
// column is NaN at the end, the split's values of that column are looked through
// again, and what is not finite among them takes its place (an infinity where
// all have one sign).  In a row of finite scores that is what the definition
// gives, for either copy: the row meets all of these keys.
template <int D, int TILES, bool HALVES>
__global__ void __launch_bounds__(128 * (TILES + 1), 1)
    fa_prefix_kernel(const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmP, const PagedParams p) {
    using T = PrefixTraits<D, TILES>;
    static_assert(!HALVES || TILES == 1, "one tile holds both copies");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bar_q = reinterpret_cast<uint64_t*>(smem + T::BAR_OFF);
    uint64_t* full = bar_q + 1;
    uint64_t* empty = full + T::NSLOT;
    uint64_t* s_full = empty + T::NSLOT;
    uint64_t* p_ready = s_full + 2;
    uint64_t* o_final = p_ready + 2;
    uint64_t* o_done = o_final + 2;
    uint64_t* v_last = o_done + 1;
    uint64_t* v_fixed = v_last + 1;
    uint64_t* mma_done = v_fixed + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + T::MISC_OFF + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Row tiles fastest: CTAs that read the same keys run together.
    int idx = blockIdx.x;
    const int rt = idx % p.row_tiles;
    idx /= p.row_tiles;
    const int split = idx % p.prefix_splits;
    const int head = idx / p.prefix_splits;
    const int r0 = rt * 128 * TILES;
    const int kbeg = split * p.prefix_chunk;
    const int kend = min(kbeg + p.prefix_chunk, p.prefix_len);
    const int nblk = (kend - kbeg + T::BN - 1) / T::BN;  // >= 1 by the host's plan
    const int tail = (kend - kbeg) & (T::BN - 1);        // keys of a partial last block

    if (threadIdx.x == 0) {
        mbar_init(bar_q, 128 * TILES);
        for (int s = 0; s < T::NSLOT; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_ready[t], 128);
            mbar_init(&o_final[t], 1);
        }
        mbar_init(o_done, 1);
        mbar_init(v_last, 1);
        mbar_init(v_fixed, 32);
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == T::MMA_WARP) {
        tmem_alloc(tmem_slot, T::TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == T::LOAD_WARP && lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        tma_prefetch_desc(&tmP);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // What was enqueued before this call ends here; the own-rows grid does not
    // depend on this one and may start then.
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t tmem = *tmem_slot;
    const AbortState st{abort_flag, p.err};
    if (warp >= 4 * TILES) {
      if constexpr (TILES == 2) setmaxnreg_dec<T::REG_CONTROL>();
      if (warp == T::LOAD_WARP) {
        // ------------------------------------------------ TMA producer
        // Lane (box, chunk) loads its part of every block; the page of the
        // next block is read while this one's slots are awaited.
        const int box = 1 << p.box_shift;
        const int lanes = (T::BN >> p.box_shift) * T::CHUNKS;
        const int b = lane / T::CHUNKS, c = lane % T::CHUNKS;
        auto key_of = [&](int j) { return kbeg + j * T::BN + (b << p.box_shift); };
        auto wants = [&](int j) { return lane < lanes && j < nblk && key_of(j) < kend; };
        int page = wants(0) ? p.prefix_pages[key_of(0) >> p.page_shift] : 0;
        // The last V of a split with a tail completes on a barrier of its own:
        // the warp that clears it waits for that one phase only.
        auto full_of = [&](int x) {
            return tail && x == 2 * nblk - 1 ? v_last : &full[x % T::NSLOT];
        };
        bool ok = true;
        int issued = 0;
        const uint64_t policy = l2_policy(p.row_tiles == 1);
        for (int j = 0; j < nblk && ok; ++j) {
            const bool mine = wants(j);
            const int z = mine ? page_plane(p, page, head) : 0;
            const int y = key_of(j) & ((1 << p.page_shift) - 1);
            const int boxes = min(T::BN >> p.box_shift,
                                  (kend - kbeg - j * T::BN + box - 1) >> p.box_shift);
            if (wants(j + 1)) page = p.prefix_pages[key_of(j + 1) >> p.page_shift];
            for (int h = 0; h < 2; ++h) {  // K_j, V_j
                const int slot = issued % T::NSLOT;
                ok = __all_sync(0xffffffffu,
                                mbar_wait(&empty[slot], ((issued / T::NSLOT) & 1) ^ 1u, st));
                if (!ok) break;
                uint64_t* bar = full_of(issued);
                if (lane == 0)
                    mbar_arrive_expect_tx(
                        bar, static_cast<uint32_t>(boxes) * box * T::CHUNKS * 128u);
                __syncwarp();
                if (mine)
                    tma_load_3d_hint(smem + T::KV_OFF + slot * T::TILE_BYTES +
                                         c * T::CHUNK_BYTES + (b << p.box_shift) * 128,
                                     h ? &tmV : &tmK, bar, c * 64, y, z, policy);
                ++issued;
            }
        }
        if (!ok)  // let the copies already requested land before exiting
            for (int x = max(0, issued - T::NSLOT); x < issued; ++x)
                mbar_wait_bounded(full_of(x),
                                  full_of(x) == v_last ? 0 : (x / T::NSLOT) & 1);
      } else if (warp == T::FIX_WARP) {
        // ------------------------------------------------ value rows behind the last key
        if (tail) {
            if (__all_sync(0xffffffffu, mbar_wait(v_last, 0, st))) {
                uint8_t* v = smem + T::KV_OFF + ((2 * nblk - 1) % T::NSLOT) * T::TILE_BYTES;
                const int units = (T::BN - tail) * 8;  // 16 bytes each, per chunk
                for (int i = lane; i < units * T::CHUNKS; i += 32)
                    *reinterpret_cast<uint4*>(v + (i / units) * T::CHUNK_BYTES + tail * 128 +
                                              (i % units) * 16) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                mbar_arrive(v_fixed);
            }
        }
      } else if (warp == T::MMA_WARP) {
        // ------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t q_base = smem_u32(smem + T::Q_OFF);
            const uint64_t dk_base = sdesc_sw128(smem_u32(smem + T::KV_OFF), 16, 1024);
            const uint64_t dv_base =
                sdesc_sw128(smem_u32(smem + T::KV_OFF), T::CHUNK_BYTES, 1024);
            // S = Q_t K^T into score buffer `buf`.
            auto mma_s = [&](int t, int buf, uint32_t slot) {
                const uint64_t a0 = sdesc_sw128(q_base + t * T::TILE_BYTES, 16, 1024);
                const uint64_t b0 = sdesc_add(dk_base, slot * T::TILE_BYTES);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k >> 2) * T::CHUNK_BYTES + (k & 3) * 32;
                    if (k == 0)
                        umma_ss_c<false>(tmem + 128u * buf, a0, b0, T::IDESC_S);
                    else
                        umma_ss_c<true>(tmem + 128u * buf, sdesc_add(a0, off), sdesc_add(b0, off),
                                        T::IDESC_S);
                }
                umma_commit(&s_full[buf]);
            };
            // O_t += P V with P in score buffer `buf`; 16 keys per step.
            auto mma_pv = [&](int t, int buf, uint32_t slot, bool acc) {
                const uint64_t b0 = sdesc_add(dv_base, slot * T::TILE_BYTES);
#pragma unroll
                for (int k = 0; k < T::BN / 16; ++k)
                    umma_ts(tmem + 256u + D * t, tmem + 128u * buf + 8u * k,
                            sdesc_add(b0, k * 2048), T::IDESC_PV, (k > 0 || acc) ? 1u : 0u);
            };
            auto wait_v = [&](int j) {
                const int x = 2 * j + 1;
                if (tail && j == nblk - 1) return mbar_wait(v_fixed, 0, st);
                return mbar_wait(&full[x % T::NSLOT], (x / T::NSLOT) & 1, st);
            };
            bool ok = mbar_wait(bar_q, 0, st);
            tc_fence_after();
            for (int j = 0; j <= nblk && ok; ++j) {
                const uint32_t ks = (2 * j) % T::NSLOT;
                const uint32_t vs = (2 * j + T::NSLOT - 1) % T::NSLOT;  // V of block j - 1
                if (j < nblk) {
                    ok = mbar_wait(&full[ks], (2 * j / T::NSLOT) & 1, st);
                    if (!ok) break;
                    tc_fence_after();
                }
                if constexpr (TILES == 1) {
                    if (j < nblk) {
                        mma_s(0, j & 1, ks);
                        umma_commit(&empty[ks]);
                    }
                    if (j > 0) {
                        const int i = j - 1;
                        ok = wait_v(i) && mbar_wait(&p_ready[i & 1], (i >> 1) & 1, st);
                        if (!ok) break;
                        tc_fence_after();
                        mma_pv(0, i & 1, vs, i > 0);
                        umma_commit(&empty[vs]);
                        umma_commit(o_done);
                        if (i == nblk - 1) umma_commit(&o_final[0]);
                    }
                } else {
                    if (j > 0 && !(ok = wait_v(j - 1))) break;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (j > 0) {
                            ok = mbar_wait(&p_ready[t], (j - 1) & 1, st);
                            if (!ok) break;
                            tc_fence_after();
                            mma_pv(t, t, vs, j > 1);
                            if (t == 1) umma_commit(&empty[vs]);
                            if (j == nblk) umma_commit(&o_final[t]);
                        }
                        if (j < nblk) mma_s(t, t, ks);
                    }
                    if (ok && j < nblk) umma_commit(&empty[ks]);
                }
            }
            // No MMA may still be running when TMEM is released.
            umma_commit(mma_done);
            mbar_wait_bounded(mma_done, 0);
        }
        __syncwarp();
      }
    } else {
        // ------------------------------------------------ softmax warpgroups
        if constexpr (TILES == 2) setmaxnreg_inc<T::REG_SOFTMAX>();
        const int t = warp >> 2, lg = warp & 3;
        const int half = HALVES ? lg >> 1 : 0;
        // This warp's first query row.
        const int wrow0 = HALVES ? (lg & 1) * 32 : r0 + 128 * t + lg * 32;
        const int row = wrow0 + lane;
        // Query rows of the warp into the swizzled tile (rows past R: zeros),
        // all copies in flight at once: through registers, four at a time, this
        // took 9 us of cold reads.
        {
            constexpr int LPR = D / 8;  // lanes per row
            const uint32_t qt = smem_u32(smem + T::Q_OFF + t * T::TILE_BYTES);
            const int u = lane % LPR;
#pragma unroll 4
            for (int i = 0; i < LPR; ++i) {
                const int rr = i * (32 / LPR) + lane / LPR;
                const int r = min(wrow0 + rr, p.R - 1), local = lg * 32 + rr;
                const int tok = r / p.G;
                const long long at =
                    (static_cast<long long>(tok) * p.Hq + head * p.G + (r - tok * p.G)) * D;
                cp_async16(qt + (u >> 3) * T::CHUNK_BYTES + sw128_offset(local, u & 7),
                           p.q + at + 8 * u, wrow0 + rr < p.R ? 16u : 0u);
            }
            cp_async_wait_all();
            fence_proxy_async_smem();
            mbar_arrive(bar_q);
        }
        const bool live = wrow0 < p.R;  // any row of this warp is a query row
        const uint32_t lane_off = static_cast<uint32_t>(lg * 32) << 16;
        const uint32_t o_tm = tmem + lane_off + 256u + D * t;
        const float sl2 = p.scale_log2;
        float m = -INFINITY, l = 0.f, lr = 0.f;
        bool ok = true;
        for (int j = 0; j < nblk; ++j) {
            const int buf = TILES == 2 ? t : (j & 1);
            const uint32_t par = TILES == 2 ? (j & 1) : ((j >> 1) & 1);
            const uint32_t s_tm = tmem + lane_off + 128u * buf;
            ok = __all_sync(0xffffffffu, mbar_wait(&s_full[buf], par, st));
            if (!ok) break;
            tc_fence_after();
            if (live) {
                constexpr int NC = HALVES ? 64 : 128;  // this thread's keys of the block
                uint32_t sr[NC / 32][32];
#pragma unroll
                for (int c = 0; c < NC / 32; ++c)
                    tmem_ld32(s_tm + 64u * half + 32u * c, sr[c]);
                tmem_ld_wait();
                if (tail && j == nblk - 1) {
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        if (c + 64 * half >= tail) sr[c >> 5][c & 31] = __float_as_uint(-INFINITY);
                }
                float mx[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) mx[i] = __uint_as_float(sr[0][i]);
#pragma unroll
                for (int c = 8; c < NC; c += 8)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mx[i] = fmaxf(mx[i], __uint_as_float(sr[(c + i) >> 5][(c + i) & 31]));
                mx[0] = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                              fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
                const float m_blk = mx[0] * sl2;
                const float m_new = m_blk > m + T::TAU ? m_blk : m;
                if (j > 0) {
                    const bool grow = m_new != m;
                    if (__any_sync(0xffffffffu, grow)) {
                        // One tile: this block's scores were issued ahead of
                        // the previous block's P V, which must be done with O.
                        if (TILES == 1) {
                            ok = __all_sync(0xffffffffu, mbar_wait(o_done, (j - 1) & 1, st));
                            if (!ok) break;
                            tc_fence_after();
                        }
                        const float alpha = grow ? ex2_approx(m - m_new) : 1.0f;
                        l *= alpha;
                        lr *= alpha;
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(o_tm + 32u * c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st32(o_tm + 32u * c, o);
                        }
                    }
                }
                m = m_new;
                // Weights exp2(s * scale*log2(e) - m), rounded to bf16 for
                // P V; l sums them unrounded (for the LSE), lr rounded (so O
                // is normalised by the weights the MMA used).
                const float mm = m == -INFINITY ? 0.f : m;
                const uint64_t sl2x2 = f2_pack(sl2, sl2), negm2 = f2_pack(-mm, -mm);
                uint64_t sum2[2] = {0ull, 0ull};
                float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < NC / 64; ++h) {
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int c = 64 * h + 2 * e;
                        float x0, x1;
                        f2_unpack(ffma2(f2_pack(__uint_as_float(sr[c >> 5][c & 31]),
                                                __uint_as_float(sr[c >> 5][(c & 31) + 1])),
                                        sl2x2, negm2),
                                  x0, x1);
                        const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                        sum2[e & 1] = fadd2(sum2[e & 1], f2_pack(p0, p1));
                        pk[e] = pack_bf16x2(p0, p1);
                        add_bf16x2_to_f32(pk[e], rs[2 * (e & 1)], rs[2 * (e & 1) + 1]);
                    }
                    tmem_st32(s_tm + 32u * (h + half), pk);
                }
                if constexpr (HALVES) {  // the other copy's keys weigh nothing here
                    uint32_t zero[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) zero[e] = 0u;
                    tmem_st32(s_tm + 32u * (1 - half), zero);
                }
                float a0, a1;
                f2_unpack(fadd2(sum2[0], sum2[1]), a0, a1);
                l += a0 + a1;
                lr += (rs[0] + rs[1]) + (rs[2] + rs[3]);
                tmem_st_wait();
            }
            tc_fence_before();
            mbar_arrive(&p_ready[buf]);
        }
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&o_final[t], 0, st));
        if (ok && live) {
            tc_fence_after();
            const bool none = l == 0.f;  // (a NaN score leaves l a NaN)
            const float inv = none ? 0.f : 1.f / lr;
            const int plane = (HALVES ? 2 * split + half : split) * p.Hkv + head;
            // O (fp32) leaves 32 columns at a time through this warp's rows of
            // the query tile, which no MMA reads any more.
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint8_t* stage = smem + T::Q_OFF + t * T::TILE_BYTES +
                                 (c % T::CHUNKS) * T::CHUNK_BYTES + lg * 32 * 128;
                uint32_t o[32];
                tmem_ld32(o_tm + 32u * c, o);
                tmem_ld_wait();
                if constexpr (HALVES) {
                    static_assert(D == 64, "two columns a lane");
                    bool bad = false;
#pragma unroll
                    for (int e = 0; e < 32; ++e) bad |= isnan(__uint_as_float(o[e]));
                    // (a row with a NaN score stays NaN: its sum is one)
                    if (__any_sync(0xffffffffu, bad && !isnan(l))) {
                        const float2 f =
                            not_finite_values(p.v_pages, p.prefix_pages, p.num_pages, p.Hkv, head,
                                              p.page_shift, kbeg, kend);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float x =
                                __shfl_sync(0xffffffffu, e & 1 ? f.y : f.x, 16 * c + e / 2);
                            if (isnan(__uint_as_float(o[e]))) o[e] = __float_as_uint(x);
                        }
                    }
                }
                if (c >= T::CHUNKS) {  // the store that used this buffer has read it
                    if (lane == 0) bulk_wait_group_read<T::CHUNKS - 1>();
                    __syncwarp();
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    uint4 v;
                    v.x = __float_as_uint(__uint_as_float(o[4 * u + 0]) * inv);
                    v.y = __float_as_uint(__uint_as_float(o[4 * u + 1]) * inv);
                    v.z = __float_as_uint(__uint_as_float(o[4 * u + 2]) * inv);
                    v.w = __float_as_uint(__uint_as_float(o[4 * u + 3]) * inv);
                    *reinterpret_cast<uint4*>(stage + sw128_offset(lane, u)) = v;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&tmP, stage, c * 32, wrow0, plane);
                    bulk_commit_group();
                }
            }
            if (lane == 0) bulk_wait_group0();
            if (row < p.R)
                p.part_lse[static_cast<long long>(plane) * p.R + row] =
                    none ? -INFINITY : m + log2f(l);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == T::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, T::TMEM_COLS);
    }
}

// ------------------------------------------------------------------ own rows

template <int D, int NR>
struct OwnTraits {
    static constexpr int ROWS = NR;  // query rows per tile
    static constexpr int BK = 64;    // keys per stage, 16 per warp
    static constexpr int NCW = 4;    // consumer warps
    static constexpr int CHUNKS = D / 64;
    static constexpr int CHUNK_BYTES = BK * 128;
    static constexpr int TILE_BYTES = BK * D * 2;
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
    static constexpr int NSTAGE = D == 128 ? 3 : 4;
    static constexpr int THREADS = (NCW + 1) * 32;
    static constexpr int BAR_OFF = NSTAGE * STAGE_BYTES;
    static constexpr int ML_OFF = BAR_OFF + 2 * NSTAGE * 8;      // [NCW][ROWS][3]
    static constexpr int SCAN_OFF = ML_OFF + NCW * ROWS * 3 * 4;  // see line_start
    static constexpr int MISC_OFF = SCAN_OFF + 64;
    static constexpr int SMEM_BYTES = MISC_OFF + 16 + 1024;
    static constexpr int MIN_CTAS = D == 128 ? 2 : 3;
    static_assert(SCAN_OFF % 8 == 0, "alignment");
    // The four warps' results meet in the last stage of their tile.
    static_assert(NCW * ROWS * D * 4 <= STAGE_BYTES, "merge buffer exceeds a stage");
};

// a / b of numbers that are not negative; a 32-bit division takes a fifth of
// the time.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// One sequence of the line, or (s = S) the prefix as seen by all T tokens.
struct LineSeq {
    int start, n, len, tiles, blocks;  // first token, tokens, keys, row tiles, key blocks
    __device__ __forceinline__ int span() const { return blocks + kLineTileBlocks; }  // a tile's

    __device__ __forceinline__ LineSeq() {}
    __device__ __forceinline__ LineSeq(const PagedParams& p, int s) {
        if (s == p.S) {
            start = 0;
            n = p.prefix_in_line ? p.T : 0;
            len = p.prefix_len;
        } else {
            start = max(0, min(p.seq_start[s], p.T));
            n = max(start, min(p.seq_start[s + 1], p.T)) - start;
            const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
            len = static_cast<int>(
                max(0ll, min(static_cast<long long>(p.kv_len[s]), cap)));
        }
        tiles = static_cast<int>((static_cast<long long>(n) * p.G + p.tile_rows - 1) / p.tile_rows);
        blocks = max(1, (len + 63) / 64);  // a tile without keys still has to be written
    }
    __device__ __forceinline__ long long size(const PagedParams& p) const {
        return static_cast<long long>(tiles) * p.Hkv * span();
    }
};

// A tile's share of a CTA: blocks [b0, b1) of row tile rt of (sequence s, head).
// The line runs over sequences, heads, row tiles (they share keys) and a
// tile's key blocks and its fixed cost; a CTA that would begin with the latter
// begins with the next tile.
struct LineWalk {
    LineSeq seq;
    int s, head, rt, b0, b1;
    long long left;  // blocks that the CTA still has, this share's not counted

    __device__ __forceinline__ LineWalk(const PagedParams& p, int s0, long long rem,
                                        long long quota)
        : seq(p, s0), s(s0), left(quota) {
        const long long tile = quotient(rem, seq.span());
        b0 = static_cast<int>(rem - tile * seq.span());
        head = static_cast<int>(quotient(tile, seq.tiles));
        rt = static_cast<int>(tile - static_cast<long long>(head) * seq.tiles);
        take();
    }
    __device__ __forceinline__ bool empty() const { return b0 >= seq.blocks; }
    __device__ __forceinline__ bool whole() const { return b0 == 0 && b1 >= seq.blocks; }
    __device__ __forceinline__ void take() {
        b1 = static_cast<int>(min(static_cast<long long>(seq.span()), b0 + left));
        left -= b1 - b0;
    }
    // To the next share; false at the end of the CTA's blocks or of the line.
    __device__ __forceinline__ bool next(const PagedParams& p) {
        if (left <= 0) return false;
        b0 = 0;
        if (++rt == seq.tiles) {
            rt = 0;
            if (++head == p.Hkv) {
                head = 0;
                do {
                    if (++s > p.S) return false;
                    seq = LineSeq(p, s);
                } while (seq.tiles == 0);
            }
        }
        take();
        return true;
    }
    // Keys [first, second) of this share that the tile's last token sees.
    __device__ __forceinline__ int2 keys(const PagedParams& p) const {
        int seen = seq.len;
        if (s < p.S) {
            const int last = (min((rt + 1) * p.tile_rows, seq.n * p.G) - 1) / p.G;
            seen = max(0, min(seq.len, seq.len - seq.n + last + 1));
        }
        const int beg = min(b0 * 64, seen);
        return make_int2(beg, min(b1 * 64, seen));
    }
};

// Where this CTA's share of the line begins: sequence `s`, block `rem` of it.
// All threads sum the sequences' sizes (contiguous runs of them); false: the
// CTA has none.  scan: 8 long longs of shared memory.
template <int THREADS>
__device__ __forceinline__ bool line_start(const PagedParams& p, long long* scan, int& s,
                                           long long& rem, long long& quota) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int count = p.S + 1, per = (count + THREADS - 1) / THREADS;
    const int a = min(count, static_cast<int>(threadIdx.x) * per), z = min(count, a + per);
    long long sum = 0;
#pragma unroll 4
    for (int i = a; i < z; ++i) sum += LineSeq(p, i).size(p);
    long long upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    long long total = 0, before = upto - sum;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    quota = max(static_cast<long long>(kLineMinBlocks), quotient(total + gridDim.x - 1, gridDim.x));
    const long long pos = blockIdx.x * quota;
    __syncthreads();
    if (pos >= before && pos < before + sum) {
        long long at = before;
        for (int i = a; i < z; ++i) {
            const long long size = LineSeq(p, i).size(p);
            if (pos >= at && pos < at + size) {
                scan[0] = i;
                scan[1] = pos - at;
            }
            at += size;
        }
    }
    __syncthreads();
    s = static_cast<int>(scan[0]);
    rem = scan[1];
    return pos < total;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of bf16, two values of a row in each lane, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Either bf16 of a pair is an infinity or a NaN.
__device__ __forceinline__ bool not_finite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// o0 (columns col, col + 1 of rows rq and rq + 8) and o1 (columns col + 8,
// + 9) += P V over the 16 keys from row `r` of the V tile, each row taking the
// keys that it sees and no others.  pa: the weights as an mma's A fragment.
template <int CHUNK_BYTES>
__device__ __noinline__ void add_visible_row(const uint8_t* v, int r, int col, uint32_t w0,
                                             uint32_t w1, int j0, int end0, int end1,
                                             float (&o)[8]) {
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
        const int src = (threadIdx.x & 28) | (e >> 1);
        const uint32_t a = __shfl_sync(0xffffffffu, w0, src), b = __shfl_sync(0xffffffffu, w1, src);
        const float p0 = __uint_as_float(e & 1 ? a & 0xffff0000u : a << 16);
        const float p1 = __uint_as_float(e & 1 ? b & 0xffff0000u : b << 16);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = col + 8 * h;
            const uint32_t x = *reinterpret_cast<const uint32_t*>(
                v + (c >> 6) * CHUNK_BYTES + sw128_offset(r + e, (c & 63) >> 3) + (c & 7) * 2);
            const float x0 = __uint_as_float(x << 16), x1 = __uint_as_float(x & 0xffff0000u);
            if (j0 + e < end0) {
                o[4 * h] += p0 * x0;
                o[4 * h + 1] += p0 * x1;
            }
            if (j0 + e < end1) {
                o[4 * h + 2] += p1 * x0;
                o[4 * h + 3] += p1 * x1;
            }
        }
    }
}
// The same for the transposed products: o = values col and col + 8 of the two
// rows whose weights for key e of eight lie in lane 4 e + cq, packed in w0 (the
// first eight keys) and w1.
template <int CHUNK_BYTES>
__device__ __noinline__ void add_visible8(const uint8_t* v, int r, int col, uint32_t w0,
                                          uint32_t w1, int j0, int end0, int end1,
                                          float (&o)[4]) {
#pragma unroll 1
    for (int e = 0; e < 16; ++e) {
        const uint32_t w =
            __shfl_sync(0xffffffffu, e < 8 ? w0 : w1, ((e & 7) << 2) | (threadIdx.x & 3));
        const float p0 = __uint_as_float(w << 16), p1 = __uint_as_float(w & 0xffff0000u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = col + 8 * h;
            const float x = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(
                v + (c >> 6) * CHUNK_BYTES + sw128_offset(r + e, (c & 63) >> 3) + (c & 7) * 2));
            if (j0 + e < end0) o[2 * h] += p0 * x;
            if (j0 + e < end1) o[2 * h + 1] += p1 * x;
        }
    }
}
template <int CHUNK_BYTES>
__device__ __forceinline__ void add_visible(const uint8_t* v, int r, int col,
                                            const uint32_t (&pa)[4], const int (&lim)[2], int j0,
                                            int kend, float (&o0)[4], float (&o1)[4]) {
    float o[8] = {o0[0], o0[1], o0[2], o0[3], o1[0], o1[1], o1[2], o1[3]};
    const int end0 = min(lim[0] + 1, kend), end1 = min(lim[1] + 1, kend);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        add_visible_row<CHUNK_BYTES>(v, r + 8 * i, col, pa[2 * i], pa[2 * i + 1], j0 + 8 * i, end0,
                                     end1, o);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        o0[e] = o[e];
        o1[e] = o[4 + e];
    }
}

// One CTA: an equal share of the line, tile after tile.  Row r of a sequence is
// head r % G of its new token r / G.  Each of four warps takes 16 keys of every
// 64-key stage and keeps its own running maximum, sum and O; they are merged
// at the end of a tile's share.
//
// Bound by HBM where sequences are long: 16 of 8192 keys, 16 heads of 128: 164
// to 169 us for 1.07 GB (97 to 100 % of the measured copy bandwidth).  Ragged
// short sequences pay the first 6 us, in which the lengths, page table and first
// stages come in one after another, and a tile's fixed part (its rows, joining
// the warps, writing); 64 sequences of 512 keys on average, 8 heads of 128,
// behind a prefix: 26 us for 134 MB.
//
// Up to 8 rows (NR = 8) the products are transposed: S^T = K Q^T and O^T =
// V^T P^T have the keys, or the head's values, along the 16 rows of an mma and
// the queries along its 8 columns, so that none of it multiplies padding: half
// the MMAs and half the registers for Q and O.  P^T is moved from one operand
// layout to the other by movmatrix, and the rows' maxima are looked at by a
// vote, and reduced only when one has risen.  (16 rows: 1.25 us for a 64-key
// stage of a CTA, 3.3 us for a tile; that case 30 us.)
//
// Weights are rounded to bf16, the type of V, because an mma multiplies two
// operands of one 16-bit type: the error of O against 64 bits is 0.0023 of its
// norm, where rounding O alone leaves 0.0017.  To keep more of a weight would take
// a second product with what the first leaves.  Scores, maxima, sums (of the
// rounded weights for O, of the unrounded for the log-sum-exp) and partial
// results are fp32.
template <int D, int NR>
__global__ void __launch_bounds__(OwnTraits<D, NR>::THREADS, OwnTraits<D, NR>::MIN_CTAS)
    fa_own_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const PagedParams p) {
    using T = OwnTraits<D, NR>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + T::BAR_OFF);
    uint64_t* empty = full + T::NSTAGE;
    float* red_ml = reinterpret_cast<float*>(smem + T::ML_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + T::MISC_OFF);
    volatile int* carry_on = abort_flag + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < T::NSTAGE; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], T::NCW);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    // Behind a prefix this grid starts when the prefix's has seen the end of
    // what came before; alone it waits for that itself (see launch_overlapped).
    if (!p.prefix_splits) grid_dependency_wait();
    grid_launch_dependents();
    // Starts, lengths and counts out of range are reported once.
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < p.S; i += T::THREADS) {
            const LineSeq q(p, i);
            const int a = p.seq_start[i], z = p.seq_start[i + 1];
            if (a < 0 || z < a || z > p.T ||
                (q.n > 0 && (p.kv_len[i] != q.len || q.n > p.max_new)))
                atomicOr(p.err, kErrIndex);
        }
    int s0;
    long long rem, quota;
    const bool any = line_start<T::THREADS>(p, reinterpret_cast<long long*>(smem + T::SCAN_OFF),
                                            s0, rem, quota);
    // The merge waits for this grid only, so this grid ends after the prefix
    // grid (which it was allowed to overtake): its first CTA waits for that, at
    // its end, and keeps no other from its place.
    auto leave = [&] {
        if (blockIdx.x == 0 && p.prefix_splits) grid_dependency_wait();
    };
    if (!any) {
        leave();
        return;
    }
    const AbortState st{abort_flag, p.err};
    LineWalk walk(p, s0, rem, quota);
    if (walk.empty() && !walk.next(p)) {
        leave();
        return;
    }

    if (warp == T::NCW) {
        // ------------------------------------------------ producer
        const int box = 1 << p.box_shift, nb = T::BK >> p.box_shift;
        const int b = lane / (2 * T::CHUNKS), c = (lane >> 1) % T::CHUNKS, h = lane & 1;
        int issued = 0;
        bool ok = true;
        do {
            const int2 keys = walk.keys(p);
            const int nblk = (keys.y - keys.x + T::BK - 1) / T::BK;
            auto key_of = [&](int j) { return keys.x + j * T::BK + (b << p.box_shift); };
            auto wants = [&](int j) { return b < nb && j < nblk && key_of(j) < keys.y; };
            const int* table = walk.s == p.S ? p.prefix_pages
                                             : p.block_table +
                                                   static_cast<long long>(walk.s) * p.max_pages;
            int page = wants(0) ? table[key_of(0) >> p.page_shift] : 0;
            // Keys of one row tile are read once: they leave L2 before the
            // partial results that the merge will read.
            const uint64_t policy = l2_policy(walk.seq.tiles == 1);
            for (int j = 0; j < nblk && ok; ++j) {
                const int slot = issued % T::NSTAGE;
                const bool mine = wants(j);
                const int z = mine ? page_plane(p, page, walk.head) : 0;
                const int y = key_of(j) & ((1 << p.page_shift) - 1);
                const int boxes = min(nb, (keys.y - keys.x - j * T::BK + box - 1) >> p.box_shift);
                if (wants(j + 1)) page = table[key_of(j + 1) >> p.page_shift];
                ok = __all_sync(0xffffffffu,
                                mbar_wait(&empty[slot], ((issued / T::NSTAGE) & 1) ^ 1u, st));
                if (!ok) break;
                if (lane == 0)
                    mbar_arrive_expect_tx(&full[slot],
                                          static_cast<uint32_t>(boxes) * box * T::CHUNKS * 256u);
                __syncwarp();
                if (mine)
                    tma_load_3d_hint(smem + slot * T::STAGE_BYTES + h * T::TILE_BYTES +
                                         c * T::CHUNK_BYTES + (b << p.box_shift) * 128,
                                     h ? &tmV : &tmK, &full[slot], c * 64, y, z, policy);
                ++issued;
            }
        } while (ok && walk.next(p));
        // Do not leave with copies in flight.
        for (int j = max(0, issued - T::NSTAGE); j < issued; ++j)
            mbar_wait_bounded(&full[j % T::NSTAGE], (j / T::NSTAGE) & 1);
        leave();
        return;
    }

    // ---------------------------------------------------- consumers
    const int rq = lane >> 2, cq = lane & 3;  // fragment row and column group
    // This warp's 16 keys of a stage: ldmatrix row of each lane.
    const int key_k = 16 * warp + ((lane >> 4) << 3) + (lane & 7);  // K: keys by matrix pair
    const int unit_k = (lane >> 3) & 1;
    const int key_v = 16 * warp + (((lane >> 3) & 1) << 3) + (lane & 7);
    const int unit_v = lane >> 4;
    int done = 0;  // stages read so far
    bool ok = true, first = true;
    do {
        const LineSeq& seq = walk.seq;
        const int start = seq.start, n = seq.n, len = seq.len, head = walk.head;
        const int rows = n * p.G, r0 = walk.rt * T::ROWS;
        const bool prefix = walk.s == p.S;
        const int2 keys = walk.keys(p);
        const int kbeg = keys.x, kend = keys.y, nblk = (kend - kbeg + T::BK - 1) / T::BK;
        // Row r of the tile: its output row, and its row among the partials.
        auto out_row = [&](int r) {
            const int i = (r0 + r) / p.G;
            return static_cast<long long>(start + i) * p.Hq + head * p.G + (r0 + r - i * p.G);
        };
        const bool whole = walk.whole();
        const bool direct = whole && p.prefix_len == 0;
        const long long part0 =
            whole ? (static_cast<long long>(prefix ? 0 : p.slots - 1) * p.Hkv + head) * p.R +
                        static_cast<long long>(start) * p.G + r0
                  : p.piece_row + (2ll * blockIdx.x + (first ? 0 : 1)) * kPieceRows;
        if (walk.b0 == 0 && threadIdx.x < T::ROWS && r0 + static_cast<int>(threadIdx.x) < rows) {
            // The tile's later blocks are the next CTAs', `quota` for each.
            const int rest = seq.blocks - walk.b1;
            const int2 d = make_int2(
                rest <= 0 ? 1 : 2 + static_cast<int>(quotient(rest - 1, quota)),
                (2 * static_cast<int>(blockIdx.x) + (first ? 0 : 1)) * kPieceRows + threadIdx.x);
            p.pieces[(static_cast<long long>(prefix) * p.Hkv + head) * p.R +
                     static_cast<long long>(start) * p.G + r0 + threadIdx.x] = d;
        }
        first = false;
        if (nblk == 0) {
            // No key in this share: an empty partial, or the empty row's result.
            for (int i = threadIdx.x; i < T::ROWS * (D / 8); i += T::NCW * 32) {
                const int r = i / (D / 8), u = i % (D / 8);
                if (r0 + r >= rows) break;  // i rises with r
                if (direct)
                    *reinterpret_cast<uint4*>(p.o + out_row(r) * D + 8 * u) =
                        make_uint4(0u, 0u, 0u, 0u);
                if (u == 0) (direct ? p.lse[out_row(r)] : p.part_lse[part0 + r]) = -INFINITY;
            }
            continue;
        }
        int slot = 0;
        float* red;
        const int lim0 = prefix ? len : len - n + r0 / p.G;  // last key of the tile's first row
        // Last visible key of row i of the tile.
        auto last_key = [&](int i) {
            const int r = r0 + i;
            return r >= rows ? -1 : prefix ? len - 1 : min(len, len - n + r / p.G + 1) - 1;
        };
        if constexpr (NR == 8) {
            // This thread's scores: keys rq and rq + 8, rows 2 cq and 2 cq + 1.
            const int lim[2] = {last_key(2 * cq), last_key(2 * cq + 1)};
            uint32_t qb[D / 16][2];
            {
                const bool real = r0 + rq < rows;
                const __nv_bfloat16* src = p.q + (real ? out_row(rq) : 0) * D + 2 * cq;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    qb[k][0] = real ? *reinterpret_cast<const uint32_t*>(src + 16 * k) : 0u;
                    qb[k][1] = real ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8) : 0u;
                }
            }
            float o[D / 16][4];  // values 16 i + rq and + 8 of the two rows
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, lr[2] = {0.f, 0.f};
            const int key_a = 16 * warp + (lane & 15), unit_a = lane >> 4;
            const int key_t = 16 * warp + (lane & 7) + ((lane >> 4) << 3), unit_t = (lane >> 3) & 1;

            for (int j = 0; j < nblk; ++j, ++done) {
                slot = done % T::NSTAGE;
                ok = __all_sync(0xffffffffu, mbar_wait(&full[slot], (done / T::NSTAGE) & 1, st));
                if (!ok) break;
                const uint32_t kt = smem_u32(smem + slot * T::STAGE_BYTES);
                const int j0 = kbeg + j * T::BK + 16 * warp;  // the warp's first key
                if (j0 < kend) {
                    float sc[2][4];  // two chains of products
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[i][e] = 0.f;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const int u = 2 * k + unit_a;
                        uint32_t a[4];
                        ldsm4(kt + (u >> 3) * T::CHUNK_BYTES + sw128_offset(key_a, u & 7), a);
                        mma16816(sc[k & 1], a, qb[k][0], qb[k][1]);
                    }
                    float v[2][2];  // [row][key]
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int y = 0; y < 2; ++y) v[x][y] = sc[0][2 * y + x] + sc[1][2 * y + x];
                    if (j0 + 15 > lim0 || j0 + 16 > kend) {
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const int key = j0 + rq + 8 * y;
                                if (key >= kend || key > lim[x]) v[x][y] = -INFINITY;
                            }
                    }
                    float bm[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) bm[x] = fmaxf(v[x][0], v[x][1]) * p.scale_log2;
                    if (__any_sync(0xffffffffu, bm[0] > m[0] + 8.f || bm[1] > m[1] + 8.f)) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1)
                                bm[x] = fmaxf(bm[x], __shfl_xor_sync(0xffffffffu, bm[x], d));
                            if (bm[x] > m[x] + 8.f) {
                                const float alpha = ex2_approx(m[x] - bm[x]);  // 0 while m = -inf
                                l[x] *= alpha;
                                lr[x] *= alpha;
#pragma unroll
                                for (int i = 0; i < D / 16; ++i) {
                                    o[i][x] *= alpha;
                                    o[i][2 + x] *= alpha;
                                }
                                m[x] = bm[x];
                            }
                        }
                    }
                    const float mm[2] = {m[0] == -INFINITY ? 0.f : m[0],
                                         m[1] == -INFINITY ? 0.f : m[1]};
                    uint32_t w[2], pb[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float p0 = ex2_approx(fmaf(v[0][y], p.scale_log2, -mm[0]));
                        const float p1 = ex2_approx(fmaf(v[1][y], p.scale_log2, -mm[1]));
                        l[0] += p0;
                        l[1] += p1;
                        w[y] = pack_bf16x2(p0, p1);
                        add_bf16x2_to_f32(w[y], lr[0], lr[1]);
                        pb[y] = transpose8x8(w[y]);
                    }
                    // Keys 2cq, 2cq + 1 (pb[0]) and 2cq + 8, 2cq + 9 (pb[1]) behind
                    // the last one: their values count as zeros.
                    const int left = kend - j0;
                    uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
                    if (left < 16) {
                        keep0 = (2 * cq < left ? 0xffffu : 0u) |
                                (2 * cq + 1 < left ? 0xffff0000u : 0u);
                        keep1 = (2 * cq + 8 < left ? 0xffffu : 0u) |
                                (2 * cq + 9 < left ? 0xffff0000u : 0u);
                    }
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const int u = 2 * i + unit_t;
                        uint32_t a[4];
                        ldsm4t(kt + T::TILE_BYTES + (u >> 3) * T::CHUNK_BYTES +
                                   sw128_offset(key_t, u & 7),
                               a);
                        a[0] &= keep0;
                        a[1] &= keep0;
                        a[2] &= keep1;
                        a[3] &= keep1;
                        // As below: values that are not finite reach only the
                        // rows that see their key.
                        if (j0 + 15 > lim0 &&
                            __any_sync(0xffffffffu, not_finite(a[0]) || not_finite(a[1]) ||
                                                        not_finite(a[2]) || not_finite(a[3]))) {
                            float t[4] = {o[i][0], o[i][1], o[i][2], o[i][3]};
                            add_visible8<T::CHUNK_BYTES>(
                                smem + slot * T::STAGE_BYTES + T::TILE_BYTES, 16 * warp,
                                16 * i + rq, w[0], w[1], j0, min(lim[0] + 1, kend),
                                min(lim[1] + 1, kend), t);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[i][e] = t[e];
                            continue;
                        }
                        mma16816(o[i], a, pb[0], pb[1]);
                    }
                }
                __syncwarp();
                if (lane == 0 && j + 1 < nblk) mbar_arrive(&empty[slot]);
            }

            // Row sums over the eight lanes that share a row, then the four
            // warps' results through the tile's last stage, given back after
            // that, its 8-float units swapped by row pair.
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    l[x] += __shfl_xor_sync(0xffffffffu, l[x], d);
                    lr[x] += __shfl_xor_sync(0xffffffffu, lr[x], d);
                }
            red = reinterpret_cast<float*>(smem + slot * T::STAGE_BYTES);  // [NCW][ROWS][D]
            named_bar_sync(1, T::NCW * 32);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = warp * T::ROWS + 2 * cq + x;
                if (rq == 0) {
                    red_ml[3 * r] = m[x];
                    red_ml[3 * r + 1] = l[x];
                    red_ml[3 * r + 2] = lr[x];
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    red[r * D + 8 * ((2 * i) ^ cq) + rq] = o[i][x];
                    red[r * D + 8 * ((2 * i + 1) ^ cq) + rq] = o[i][2 + x];
                }
            }
        } else {
            uint32_t qa[D / 16][4];
            int lim[2];  // last visible key of rows rq and rq + 8
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = r0 + rq + 8 * x;
                lim[x] = last_key(rq + 8 * x);
                const __nv_bfloat16* src = p.q + (r < rows ? out_row(rq + 8 * x) : 0) * D + 2 * cq;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    qa[k][x] = r < rows ? *reinterpret_cast<const uint32_t*>(src + 16 * k) : 0u;
                    qa[k][x + 2] =
                        r < rows ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8) : 0u;
                }
            }
            float o[D / 8][4];
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, lr[2] = {0.f, 0.f};

            for (int j = 0; j < nblk; ++j, ++done) {
                slot = done % T::NSTAGE;
                ok = __all_sync(0xffffffffu, mbar_wait(&full[slot], (done / T::NSTAGE) & 1, st));
                if (!ok) break;
                const uint32_t kt = smem_u32(smem + slot * T::STAGE_BYTES);
                const int j0 = kbeg + j * T::BK + 16 * warp;  // the warp's first key
                if (j0 < kend) {
                    float sc[2][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[i][e] = 0.f;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const int u = 2 * k + unit_k;
                        uint32_t b[4];
                        ldsm4(kt + (u >> 3) * T::CHUNK_BYTES + sw128_offset(key_k, u & 7), b);
                        mma16816(sc[0], qa[k], b[0], b[1]);
                        mma16816(sc[1], qa[k], b[2], b[3]);
                    }
                    // Online softmax of rows rq and rq + 8 over the warp's 16 keys.
                    uint32_t pa[4];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float v[4];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int key = j0 + 8 * i + 2 * cq + e;
                                v[2 * i + e] = key < kend && key <= lim[x]
                                                   ? sc[i][2 * x + e] * p.scale_log2
                                                   : -INFINITY;
                            }
                        float bm = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
                        bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 1));
                        bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 2));
                        if (bm > m[x] + 8.f) {
                            const float alpha = ex2_approx(m[x] - bm);  // 0 while m = -inf
                            l[x] *= alpha;
                            lr[x] *= alpha;
#pragma unroll
                            for (int i = 0; i < D / 8; ++i) {
                                o[i][2 * x] *= alpha;
                                o[i][2 * x + 1] *= alpha;
                            }
                            m[x] = bm;
                        }
                        const float mm = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float p0 = ex2_approx(v[2 * i] - mm);
                            const float p1 = ex2_approx(v[2 * i + 1] - mm);
                            l[x] += p0 + p1;
                            pa[2 * i + x] = pack_bf16x2(p0, p1);
                            float a = 0.f, b = 0.f;
                            add_bf16x2_to_f32(pa[2 * i + x], a, b);
                            lr[x] += a + b;
                        }
                    }
                    // Keys 2cq, 2cq + 1 (b0) and 2cq + 8, 2cq + 9 (b1) behind the
                    // last one: their values count as zeros.
                    const int left = kend - j0;
                    uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
                    if (left < 16) {
                        keep0 = (2 * cq < left ? 0xffffu : 0u) |
                                (2 * cq + 1 < left ? 0xffff0000u : 0u);
                        keep1 = (2 * cq + 8 < left ? 0xffffu : 0u) |
                                (2 * cq + 9 < left ? 0xffff0000u : 0u);
                    }
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const int u = 2 * i + unit_v;
                        uint32_t b[4];
                        ldsm4t(kt + T::TILE_BYTES + (u >> 3) * T::CHUNK_BYTES +
                                   sw128_offset(key_v, u & 7),
                               b);
                        b[0] &= keep0;
                        b[1] &= keep1;
                        b[2] &= keep0;
                        b[3] &= keep1;
                        // A key that some rows do not see must not reach them, and a
                        // weight of zero times infinity would: such values are added
                        // row by row.
                        if (j0 + 15 > lim0 &&
                            __any_sync(0xffffffffu, not_finite(b[0]) || not_finite(b[1]) ||
                                                        not_finite(b[2]) || not_finite(b[3]))) {
                            add_visible<T::CHUNK_BYTES>(
                                smem + slot * T::STAGE_BYTES + T::TILE_BYTES, 16 * warp,
                                16 * i + 2 * cq, pa, lim, j0, kend, o[2 * i], o[2 * i + 1]);
                            continue;
                        }
                        mma16816(o[2 * i], pa, b[0], b[1]);
                        mma16816(o[2 * i + 1], pa, b[2], b[3]);
                    }
                }
                __syncwarp();
                if (lane == 0 && j + 1 < nblk) mbar_arrive(&empty[slot]);
            }

            // Row sums over the four lanes of a row, then the four warps' results
            // through the tile's last stage, which is given back only after that.  Its
            // 8-float units are swapped by row, so that the writes meet every bank.
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) {
                    l[x] += __shfl_xor_sync(0xffffffffu, l[x], d);
                    lr[x] += __shfl_xor_sync(0xffffffffu, lr[x], d);
                }
            red = reinterpret_cast<float*>(smem + slot * T::STAGE_BYTES);  // [NCW][ROWS][D]
            named_bar_sync(1, T::NCW * 32);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = warp * T::ROWS + rq + 8 * x;
                if (cq == 0) {
                    red_ml[3 * r] = m[x];
                    red_ml[3 * r + 1] = l[x];
                    red_ml[3 * r + 2] = lr[x];
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    *reinterpret_cast<float2*>(red + r * D + 8 * (i ^ (rq & 7)) + 2 * cq) =
                        make_float2(o[i][2 * x], o[i][2 * x + 1]);
            }
        }
        // One answer for all warps, so that none waits here for one that gave up.
        if (threadIdx.x == 0) *carry_on = *abort_flag == 0;
        named_bar_sync(1, T::NCW * 32);
        ok = *carry_on != 0;
        for (int i = threadIdx.x; i < T::ROWS * (D / 4); i += T::NCW * 32) {
            const int r = i / (D / 4), e4 = (i % (D / 4)) * 4;
            if (r0 + r >= rows) break;  // i rises with r
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < T::NCW; ++w) M = fmaxf(M, red_ml[3 * (w * T::ROWS + r)]);
            float L = 0.f, Lr = 0.f;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < T::NCW; ++w) {
                const float* ml = red_ml + 3 * (w * T::ROWS + r);
                // A warp that saw nothing has l = O = 0; one whose scores were all
                // NaN has m = -inf too, and its NaN must reach the row.
                const float f = ml[0] == -INFINITY ? 1.f : ex2_approx(ml[0] - M);
                const float4 x = *reinterpret_cast<const float4*>(
                    red + (w * T::ROWS + r) * D +
                    8 * ((e4 >> 3) ^ (NR == 8 ? (r >> 1) & 3 : r & 7)) + (e4 & 7));
                L += f * ml[1];
                Lr += f * ml[2];
                a.x += f * x.x;
                a.y += f * x.y;
                a.z += f * x.z;
                a.w += f * x.w;
            }
            const bool none = L == 0.f;
            const float inv = none ? 0.f : 1.f / Lr;
            const float lse2 = none ? -INFINITY : M + log2f(L);
            if (direct) {
                uint2 w;
                w.x = pack_bf16x2(a.x * inv, a.y * inv);
                w.y = pack_bf16x2(a.z * inv, a.w * inv);
                *reinterpret_cast<uint2*>(p.o + out_row(r) * D + e4) = w;
                if (e4 == 0) p.lse[out_row(r)] = lse2 * 0.6931471805599453f;
            } else {
                *reinterpret_cast<float4*>(p.part_o + (part0 + r) * D + e4) =
                    make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
                if (e4 == 0) p.part_lse[part0 + r] = lse2;
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
    } while (ok && walk.next(p));
    leave();
}

// ------------------------------------------------------------------ merge

// A row's partial results so far: O and L relative to 2^M.
template <int PER>
struct RowSum {
    float M = -INFINITY, L = 0.f, acc[PER];
    __device__ __forceinline__ RowSum() {
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = 0.f;
    }
    // Adds another sum, of the same values of the row.
    __device__ __forceinline__ void join(float M2, float L2, const float (&v)[PER]) {
        const float M1 = fmaxf(M, M2);
        const float f = M == M1 ? 1.f : ex2_approx(M - M1);
        const float f2 = M2 == M1 ? 1.f : ex2_approx(M2 - M1);
        M = M1;
        L = L * f + L2 * f2;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = acc[i] * f + v[i] * f2;
    }
    // Adds up to U partial results: O values in v, and lane x's log-sum-exp of
    // the x-th in ls.  One with nothing seen (-inf) has weight 0, and its O was
    // never written.
    template <int U>
    __device__ __forceinline__ void add(const float (&v)[U][PER], float ls) {
        float m = ls;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float M1 = fmaxf(M, m);
        const float f = M == M1 ? 1.f : ex2_approx(M - M1);
        M = M1;
        L *= f;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] *= f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float l = __shfl_sync(0xffffffffu, ls, u);
            if (l == -INFINITY) continue;
            const float w = ex2_approx(l - M);
            L += w;
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] += w * v[u][i];
        }
    }
};

// W warps per output row (token, query head): with w_x = 2^(lse_x - M) over
// the row's partial results, O = sum_x w_x O_x / sum_x w_x.  What this costs is
// its chain of dependent reads (4 us for 2048 rows of 17 results, 18 MB, behind
// the last CTA of the line; 7 while own keys pushed them out of L2), so the
// prefix's first splits, whose places are known, are read at once with the row's
// table entry, and its first pieces before any of them is added up.  Few rows
// may have many pieces (a long sequence spread over the whole GPU): the row's
// warps take them in turn.
template <int D, int W>
__global__ void __launch_bounds__(128, 5) fa_paged_merge_kernel(const PagedParams p) {
    constexpr int PER = D / 32, U = 8, V = 4;
    __shared__ float other[W > 1 ? W - 1 : 1][2 + PER][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % W;
    const long long row = static_cast<long long>(blockIdx.x) * (4 / W) + warp / W;
    const int t = static_cast<int>(row / p.Hq), hq = static_cast<int>(row - 1ll * t * p.Hq);
    const int head = hq / p.G, g = hq - head * p.G;
    grid_launch_dependents();
    // (Read ahead of the wait: when this grid may start, all that came before the
    // call has ended; see launch_overlapped.)
    const bool mine = row < static_cast<long long>(p.T) * p.Hq && t >= p.seq_start[0] &&
                      t < p.seq_start[p.S];  // else no sequence's row
    const long long plane_row = static_cast<long long>(head) * p.R +
                                static_cast<long long>(t) * p.G + g;
    const long long step = static_cast<long long>(p.Hkv) * p.R;
    grid_dependency_wait();
    if (!mine) return;
    // Where starts are out of order a row may have no tile: its values are
    // unspecified, but no read leaves the workspace.
    auto pieces_of = [&](int kind) {
        int2 d = p.pieces[kind * step + plane_row];
        d.y = max(0, min(d.y, 32 * p.line_ctas - 1));
        d.x = max(1, min(d.x, p.line_ctas - (d.y >> 5)));
        return d;
    };
    auto load = [&](float (&v)[PER], long long r) {
        const float* src = p.part_o + r * D + lane * PER;
        if constexpr (PER == 4)
            *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
        else
            *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
    };
    const int2 own = pieces_of(0);
    int2 pre = make_int2(0, 0);
    if (p.prefix_in_line) pre = pieces_of(1);
    auto load_splits = [&](int x0, float (&v)[U][PER]) {
        const int n = min(U, p.prefix_slots - x0);
        const long long r = plane_row + x0 * step;
        float ls = -INFINITY;
        if (lane < n) ls = p.part_lse[r + lane * step];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < n) load(v[u], r + u * step);
        return ls;
    };
    auto load_pieces = [&](int x0, float (&v)[V][PER]) {
        const int n = min(V, pre.x + own.x - x0);
        long long at = 0;
        float ls = -INFINITY;
        if (lane < n) {
            int x = x0 + lane;
            const bool of_own = x >= pre.x;
            const int2 d = of_own ? own : pre;
            if (of_own) x -= pre.x;
            at = d.x == 1 ? plane_row + (of_own ? p.slots - 1 : 0) * step
                          : p.piece_row + (x == 0 ? d.y : ((d.y >> 5) + x) * 32 + (d.y & 15));
            ls = p.part_lse[at];
        }
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const long long r = __shfl_sync(0xffffffffu, at, u);
            if (u < n) load(v[u], r);
        }
        return ls;
    };
    RowSum<PER> sum;
    float splits[U][PER], pieces[V][PER];
    float split_ls = load_splits(U * part, splits);
    if (p.prefix_len == 0 && own.x == 1) return;  // written by its CTA
    float piece_ls = load_pieces(V * part, pieces);
    for (int x = U * part; x < p.prefix_slots;) {
        sum.add(splits, split_ls);
        if ((x += U * W) < p.prefix_slots) split_ls = load_splits(x, splits);
    }
    for (int x = V * part; x < pre.x + own.x;) {
        sum.add(pieces, piece_ls);
        if ((x += V * W) < pre.x + own.x) piece_ls = load_pieces(x, pieces);
    }
    if constexpr (W > 1) {  // the whole block is one row's
        if (part > 0) {
            other[part - 1][0][lane] = sum.M;
            other[part - 1][1][lane] = sum.L;
#pragma unroll
            for (int i = 0; i < PER; ++i) other[part - 1][2 + i][lane] = sum.acc[i];
        }
        __syncthreads();
        if (part > 0) return;
#pragma unroll
        for (int w = 0; w < W - 1; ++w) {
            float v[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = other[w][2 + i][lane];
            sum.join(other[w][0][lane], other[w][1][lane], v);
        }
    }
    const bool none = sum.L == 0.f;
    const float inv = none ? 0.f : 1.f / sum.L;
    __nv_bfloat16* orow = p.o + row * D + lane * PER;
    if constexpr (PER == 4) {
        uint2 w;
        w.x = pack_bf16x2(sum.acc[0] * inv, sum.acc[1] * inv);
        w.y = pack_bf16x2(sum.acc[2] * inv, sum.acc[3] * inv);
        *reinterpret_cast<uint2*>(orow) = w;
    } else {
        *reinterpret_cast<uint32_t*>(orow) = pack_bf16x2(sum.acc[0] * inv, sum.acc[1] * inv);
    }
    if (lane == 0)
        p.lse[row] = none ? -INFINITY : (sum.M + log2f(sum.L)) * 0.6931471805599453f;
}

}  // namespace fa
