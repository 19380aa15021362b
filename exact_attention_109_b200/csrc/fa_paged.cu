// fa_paged.cu -- C entry points of attention over a paged cache behind a
// shared prefix (declared in include/fa.h; kernels in fa_paged_kernels.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "fa.h"
#include "fa_internal.h"
#include "fa_paged_kernels.cuh"

namespace {

using fa_host::aligned;

constexpr int kMaxDevices = 64;
// CTAs at most: they bound the workspace.
constexpr long long kMaxPrefixCtas = 512;
constexpr int kMaxLineCtas = 444;
// The figures of the rules below: microseconds of GPU time for one call, events
// around it, L2 flushed before, max_new tight; sequences of one token and 300 own
// keys unless said otherwise, pages of 64.
//
// Query rows of a key head for which the prefix joins the line of the sequences:
// a row tile of the line, and a launch less.  12 sequences behind 1024 / 16384 /
// 65536 keys, 16 heads of 64: 18 / 31 / 64 in the line, 23 / 35 / 71 on the
// tensor-core path; 16 heads of 128: 23 / 45 / 110 and 27 / 47 / 105.  32 sequences,
// 8 heads of 128, behind 1024 / 16384: 25 / 45 in the line, 26 / 38 not.
constexpr int kLinePrefixRows = 16;
// Rows of a sequence and key head up to which the line's tiles have 8.  16
// sequences of 4096 keys without a prefix, 4 heads of 128 / 64: 8 rows 37.5 / 26.6,
// in tiles of 16 39.1 / 26.7; 12 rows, which read their keys twice in tiles of 8,
// 56.9 / 32.8, and 42.7 / 27.8 in those of 16.
constexpr int kSmallTileRows = 8;
// Keys of a prefix in the line up to which two tiles of 8 rows, the second of
// which finds the keys in L2, are as good as one of 16 for it and better for the
// own keys.  16 sequences, 16 heads of 128, behind 256 / 1024 / 4096 keys: 23 / 25 /
// 31 in tiles of 8, 27 / 29 / 32 in tiles of 16; behind 16384 / 65536 keys 69 / 196
// and 48 / 111.  Heads of 64: 18 / 20 / 22.5 and 20.5 / 20.5 / 22.5, 36 / 88 and 33 / 67.
constexpr int kTwoTileKeys = 4096;
// Query rows of a key head up to which the prefix kernel takes them twice, with
// heads of 64: 20 sequences, 32 heads, behind 4096 / 16384 / 65536 keys 36 / 54 /
// 129, 38 / 60 / 148 with two idle softmax warps; 64 sequences behind 16384 75 and
// 79.  Heads of 128 are bound by HBM there (199 either way) and keep their rows once.
constexpr int kHalvesRows = 64;
// Output rows up to which the merge takes four warps for each: few rows may have
// many pieces, many rows fill the GPU anyway.  Heads of 128, four warps and one:
// 16 rows (one sequence of 37 keys) behind 1024 keys 16.4 and 18.0; 32 rows behind
// 16384 39 and 43; 16 rows of one sequence of 65536 keys 103 and 108; 1024 rows
// behind 16384 41.6 and 40.8; 2048 behind 16384, 512 own keys, 64 and 61; 4096
// behind 65536 161 and 154.
constexpr long long kWideMergeRows = 1024;

struct Plan {
    int tiles;            // query tiles per prefix CTA
    int row_tiles;        // prefix CTAs along the rows
    int prefix_splits, prefix_chunk;
    bool prefix_in_line;
    bool halves;          // the two halves of every key block apart
    int slots;            // partial results of all rows
    int line_ctas;
    int tile_rows;        // query rows of a tile of the line
};

int ilog2(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

fa_status check_sizes(int S, int T, int Hq, int Hkv, int d, int page_size, int max_pages,
                      int prefix_len, int max_new) {
    if (S < 1 || T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_pages < 1 || prefix_len < 0)
        return FA_ERR_INVALID_ARG;
    if (T > 0 && (max_new < 1 || max_new > T)) return FA_ERR_INVALID_ARG;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
        return FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (static_cast<long long>(T) * Hq > (1ll << 24) || prefix_len > (1 << 30) ||
        static_cast<long long>(max_pages) * page_size > (1ll << 30))
        return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// The prefix's tiles of query rows, and the splits that the workspace has room
// for.
Plan plan_rows(int T, int G, int Hkv, int d, int prefix_len, int max_new) {
    Plan pl{};
    const long long rows = static_cast<long long>(T) * G;
    pl.prefix_in_line = prefix_len > 0 && rows <= kLinePrefixRows;
    pl.tiles = rows > 128 ? 2 : 1;
    // A long prefix in the line is one tile, so that its keys are read once.
    const long long one_tile = pl.prefix_in_line && prefix_len > kTwoTileKeys ? rows : 0;
    pl.tile_rows =
        std::max(static_cast<long long>(max_new) * G, one_tile) <= kSmallTileRows ? 8 : 16;
    pl.halves = d == 64 && rows <= kHalvesRows;
    pl.row_tiles = static_cast<int>((rows + 128 * pl.tiles - 1) / (128 * pl.tiles));
    const long long units = static_cast<long long>(Hkv) * pl.row_tiles;
    if (prefix_len > 0 && !pl.prefix_in_line)
        pl.prefix_splits = static_cast<int>(std::min<long long>(
            (prefix_len + 127) / 128, std::max(1ll, kMaxPrefixCtas / units)));
    return pl;
}

// Partial results of the prefix for each row.
int prefix_slots(const Plan& pl) {
    return pl.prefix_in_line ? 1 : pl.prefix_splits * (pl.halves ? 2 : 1);
}

// CTAs of the line: as many as are resident, unless the longest line has less
// work.
int line_ctas(const Plan& pl, int S, int T, int G, int Hkv, int d, int page_size, int max_pages,
              int prefix_len, int max_new, int sm_count) {
    const double cap = (static_cast<long long>(max_pages) * page_size + 63) / 64;
    auto tiles = [&](long long rows) {
        return static_cast<double>((rows + pl.tile_rows - 1) / pl.tile_rows);
    };
    const double own = S * tiles(static_cast<long long>(max_new) * G) * cap;
    const double prefix = pl.prefix_in_line ? tiles(static_cast<long long>(T) * G) *
                                                  ((prefix_len + 63) / 64) : 0.0;
    const double blocks = (own + prefix) * Hkv;
    const long long per_sm =
        d == 64 ? fa::OwnTraits<64, 16>::MIN_CTAS : fa::OwnTraits<128, 16>::MIN_CTAS;
    const long long ctas = std::min<long long>(kMaxLineCtas, per_sm * sm_count);
    return blocks < ctas ? static_cast<int>(blocks) : static_cast<int>(ctas);
}

Plan make_plan(int S, int T, int Hq, int Hkv, int d, int page_size, int max_pages, int prefix_len,
               int max_new, int sm_count) {
    Plan pl = plan_rows(T, Hq / Hkv, Hkv, d, prefix_len, max_new);
    pl.line_ctas = line_ctas(pl, S, T, Hq / Hkv, Hkv, d, page_size, max_pages, prefix_len, max_new,
                             sm_count);
    if (pl.prefix_splits > 0) {
        // The splits with the fewest waves of CTAs (one per SM), a CTA's time
        // being its key blocks plus a fixed part of about three blocks' time
        // (set-up, the first loads, writing its partial result).
        const long long units = static_cast<long long>(Hkv) * pl.row_tiles;
        const long long blocks = (prefix_len + 127) / 128, most = pl.prefix_splits;
        long long best_per = 0, best_cost = 0;
        for (long long n = 0, waves = 1; n < most; ++waves) {
            n = std::min(most, std::max(1ll, waves * sm_count / units));
            const long long per = (blocks + n - 1) / n, used = (blocks + per - 1) / per;
            const long long cost = (units * used + sm_count - 1) / sm_count * (per + 3);
            if (best_per == 0 || cost < best_cost) {
                best_per = per;
                best_cost = cost;
            }
        }
        pl.prefix_splits = static_cast<int>((blocks + best_per - 1) / best_per);
        pl.prefix_chunk = static_cast<int>(best_per) * 128;
    }
    pl.slots = prefix_len == 0 ? 0 : 1 + prefix_slots(pl);
    return pl;
}

// Bytes of the table of pieces in front of the partial results.
size_t table_bytes(int T, int Hq) {
    return (static_cast<size_t>(T) * Hq * 2 * sizeof(int2) + 255) / 256 * 256;
}

// Opts the kernel into its shared memory and checks that the registers it is
// launched with cover its setmaxnreg split.
template <int D, int TILES, bool HALVES>
bool prepare_prefix() {
    using T = fa::PrefixTraits<D, TILES>;
    cudaFuncAttributes attr{};
    return cudaFuncSetAttribute(fa::fa_prefix_kernel<D, TILES, HALVES>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                T::SMEM_BYTES) == cudaSuccess &&
           cudaFuncGetAttributes(&attr, fa::fa_prefix_kernel<D, TILES, HALVES>) == cudaSuccess &&
           attr.numRegs * T::NUM_THREADS >= T::REG_BUDGET;
}
template <int D, int NR>
bool prepare_own() {
    return cudaFuncSetAttribute(fa::fa_own_kernel<D, NR>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                fa::OwnTraits<D, NR>::SMEM_BYTES) == cudaSuccess;
}

struct Ready {
    std::once_flag once;
    bool ok = false;
};
Ready g_ready[kMaxDevices];

bool prepare(int dev) {
    std::call_once(g_ready[dev].once, [&] {
        g_ready[dev].ok = prepare_prefix<64, 1, true>() && prepare_prefix<64, 1, false>() &&
                          prepare_prefix<64, 2, false>() && prepare_prefix<128, 1, false>() &&
                          prepare_prefix<128, 2, false>() &&
                          prepare_own<64, 8>() && prepare_own<64, 16>() &&
                          prepare_own<128, 8>() && prepare_own<128, 16>();
    });
    return g_ready[dev].ok;
}

template <int D>
cudaError_t launch_all(const Plan& pl, const CUtensorMap& mk, const CUtensorMap& mv,
                       const CUtensorMap& mp, const fa::PagedParams& prm, cudaStream_t s) {
    using fa_host::launch_overlapped;
    cudaError_t e = cudaSuccess;
    if (pl.prefix_splits > 0) {
        const dim3 grid(prm.Hkv * pl.row_tiles * pl.prefix_splits);
        if (pl.tiles == 2)
            e = launch_overlapped(fa::fa_prefix_kernel<D, 2, false>, grid,
                                  fa::PrefixTraits<D, 2>::NUM_THREADS,
                                  fa::PrefixTraits<D, 2>::SMEM_BYTES, s, mk, mv, mp, prm);
        else
            e = launch_overlapped(pl.halves ? fa::fa_prefix_kernel<D, 1, D == 64>
                                            : fa::fa_prefix_kernel<D, 1, false>,
                                  grid, fa::PrefixTraits<D, 1>::NUM_THREADS,
                                  fa::PrefixTraits<D, 1>::SMEM_BYTES, s, mk, mv, mp, prm);
        if (e != cudaSuccess) return e;
    }
    e = launch_overlapped(
        pl.tile_rows == 8 ? fa::fa_own_kernel<D, 8> : fa::fa_own_kernel<D, 16>,
        dim3(pl.line_ctas), fa::OwnTraits<D, 16>::THREADS,
        pl.tile_rows == 8 ? fa::OwnTraits<D, 8>::SMEM_BYTES : fa::OwnTraits<D, 16>::SMEM_BYTES, s,
        mk, mv, prm);
    if (e != cudaSuccess) return e;
    const int rows = prm.T * prm.Hq;
    return rows <= kWideMergeRows
               ? launch_overlapped(fa::fa_paged_merge_kernel<D, 4>, dim3(rows), 128, 0, s, prm)
               : launch_overlapped(fa::fa_paged_merge_kernel<D, 1>, dim3((rows + 3) / 4), 128, 0, s,
                                   prm);
}

}  // namespace

extern "C" {

size_t fa_paged_workspace_size(int S, int T, int Hq, int Hkv, int d, int page_size,
                               int max_pages, int prefix_len, int max_new) {
    if (check_sizes(S, T, Hq, Hkv, d, page_size, max_pages, prefix_len, max_new) != FA_OK ||
        T == 0)
        return 0;
    // Enough for any SM count: the splits are bounded by the sizes alone.  And for
    // any shorter prefix, which may be cut into small tiles: they make the most CTAs.
    Plan pl = plan_rows(T, Hq / Hkv, Hkv, d, prefix_len, max_new);
    pl.tile_rows = 8;
    const int ctas = line_ctas(pl, S, T, Hq / Hkv, Hkv, d, page_size, max_pages, prefix_len,
                               max_new, kMaxLineCtas);
    const size_t slots = prefix_len == 0 ? 0 : 1 + prefix_slots(pl);
    return table_bytes(T, Hq) + (slots * T * Hq + ctas * 2 * 16) * (d + 1) * sizeof(float);
}

fa_status fa_paged_split_plan(int S, int T, int Hq, int Hkv, int d, int page_size, int max_pages,
                              int prefix_len, int max_new, int sm_count, int* prefix_splits,
                              int* prefix_chunk, int* line_ctas) {
    if (!prefix_splits || !prefix_chunk || !line_ctas || sm_count < 1) return FA_ERR_INVALID_ARG;
    const fa_status st =
        check_sizes(S, T, Hq, Hkv, d, page_size, max_pages, prefix_len, max_new);
    if (st != FA_OK) return st;
    if (T == 0) return FA_ERR_INVALID_ARG;
    const Plan pl =
        make_plan(S, T, Hq, Hkv, d, page_size, max_pages, prefix_len, max_new, sm_count);
    *prefix_splits = pl.prefix_splits;
    *prefix_chunk = pl.prefix_chunk;
    *line_ctas = pl.line_ctas;
    return FA_OK;
}

fa_status fa_fwd_paged(const void* q, const void* k_pages, const void* v_pages,
                       const int* block_table, const int* seq_start, const int* kv_len,
                       const int* prefix_pages, int prefix_len, void* o, float* lse, int S, int T,
                       int Hq, int Hkv, int d, int page_size, int num_pages, int max_pages,
                       int max_new, float scale, void* workspace, size_t workspace_bytes,
                       void* stream) {
    if (!q || !k_pages || !v_pages || !block_table || !seq_start || !kv_len || !o || !lse ||
        (prefix_len > 0 && !prefix_pages))
        return FA_ERR_INVALID_ARG;
    if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
    const float sl2 = scale * 1.4426950408889634f;
    if (!(std::isfinite(sl2) && sl2 > 0.f)) return FA_ERR_INVALID_ARG;
    fa_status st = check_sizes(S, T, Hq, Hkv, d, page_size, max_pages, prefix_len, max_new);
    if (st != FA_OK) return st;
    if (num_pages < 1 || static_cast<long long>(num_pages) * Hkv >= 0x7fffffffll)
        return FA_ERR_INVALID_ARG;
    const size_t need = fa_paged_workspace_size(S, T, Hq, Hkv, d, page_size, max_pages,
                                                prefix_len, max_new);
    if (T > 0 && (!workspace || workspace_bytes < need)) return FA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(o, 16) ||
        !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(seq_start, 4) ||
        !aligned(kv_len, 4) || !aligned(prefix_pages, 4) || !aligned(workspace, 256))
        return FA_ERR_MISALIGNED;
    if (T == 0) return FA_OK;
    int dev, sms;
    unsigned int* err;
    if ((st = fa_host::device(&dev, &err, &sms)) != FA_OK) return st;
    if (!prepare(dev)) return FA_ERR_CUDA;

    const Plan pl = make_plan(S, T, Hq, Hkv, d, page_size, max_pages, prefix_len, max_new, sms);
    const size_t rows = static_cast<size_t>(pl.slots) * T * Hq;
    fa::PagedParams prm;
    prm.q = static_cast<const __nv_bfloat16*>(q);
    prm.block_table = block_table;
    prm.seq_start = seq_start;
    prm.kv_len = kv_len;
    prm.prefix_pages = prefix_pages;
    prm.v_pages = static_cast<const __nv_bfloat16*>(v_pages);
    prm.o = static_cast<__nv_bfloat16*>(o);
    prm.lse = lse;
    prm.pieces = static_cast<int2*>(workspace);
    prm.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + table_bytes(T, Hq));
    prm.part_lse = prm.part_o + (rows + pl.line_ctas * 2 * 16) * d;
    prm.piece_row = static_cast<long long>(rows);
    prm.err = err;
    prm.S = S;
    prm.T = T;
    prm.Hq = Hq;
    prm.Hkv = Hkv;
    prm.G = Hq / Hkv;
    prm.R = T * prm.G;
    prm.page_shift = ilog2(page_size);
    prm.box_shift = std::min(prm.page_shift, 6);
    prm.num_pages = num_pages;
    prm.max_pages = max_pages;
    prm.max_new = max_new;
    prm.prefix_len = prefix_len;
    prm.prefix_splits = pl.prefix_splits;
    prm.prefix_chunk = pl.prefix_chunk;
    prm.prefix_slots = pl.prefix_splits > 0 ? pl.slots - 1 : 0;
    prm.row_tiles = pl.row_tiles;
    prm.prefix_in_line = pl.prefix_in_line;
    prm.slots = pl.slots;
    prm.line_ctas = pl.line_ctas;
    prm.tile_rows = pl.tile_rows;
    prm.scale_log2 = sl2;

    const long long planes = static_cast<long long>(num_pages) * Hkv;
    const int box = 1 << prm.box_shift;
    CUtensorMap mk, mv, mp;
    if (!fa_host::encode_map(&mk, k_pages, 2, d, page_size, planes, 64, box) ||
        !fa_host::encode_map(&mv, v_pages, 2, d, page_size, planes, 64, box))
        return FA_ERR_CUDA;
    mp = mk;  // unused without a prefix
    if (pl.prefix_splits > 0 &&
        !fa_host::encode_map(&mp, prm.part_o, 4, d, prm.R,
                             static_cast<long long>(prm.prefix_slots) * Hkv, 32, 32))
        return FA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = d == 64 ? launch_all<64>(pl, mk, mv, mp, prm, s)
                                  : launch_all<128>(pl, mk, mv, mp, prm, s);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
