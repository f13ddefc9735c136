// head.cu -- token log-probabilities from hidden states and the vocabulary
// matrix, and their gradient, without keeping the logits.
//
// With x = H W^T, t near a row's largest logit and lnS = ln sum_j exp((x_j - t) it):
//   logp = (x_y - t) it - lnS,      d_ij = c_i (1[j = y_i] - p_ij),
//   dH = d W,   dW = d^T H,         c_i = L it dlogp_i.
// Rows that are left out (ignored labels; in the gradient also dlogp = 0, and rows whose logits
// are all -inf) are taken out first: the live rows' hidden states are copied together, so
// that prompts cost nothing and what such rows hold meets no product.
//
// Log-probabilities are one product whose epilogue keeps a maximum and a sum for each
// row and half tile (16 bytes for 256 logits), joined afterwards.  The gradient forms the
// logits anew, one piece of the vocabulary at a time, turns them into d, rounded to the
// operands' type, and multiplies d twice; with one piece, the usual case, that is three
// products and no sums in memory but where dH's long sum is split for the sake of idle SMs.
// A form that kept exponentials of one pass for the gradient (six products' flops instead
// of eight for a forward and a backward call) would need d scaled and rounded once more.
//
// The products are bound by the tensor cores and the power limit where they are large.
// Measured on one GB300 (cuBLAS: 1921 TFLOP/s in a burst, 1718 sustained; 6772 GB/s
// copied): log-probabilities 8192 x 50257 x 768 bf16, a quarter left out, 316 us (1500
// TFLOP/s), 4 x 32000 x 4096 bf16 55 us (4.8 TB/s: W is read once); gradient 2048 x 50257 x
// 1600 fp16, 30 % left out, 578 us (1200 TFLOP/s), 8192 x 131072 x 4096 bf16, a tenth left out,
// 15.2 ms (1560 TFLOP/s).  In the first case the tensor pipe is active in 79 % of the product's
// cycles; two SMs' tile of 256 x 256 reads 64 bytes a cycle and SM from L2 and leaves shared
// memory as many, its limit.  Rounds of tiles (the third case's are 5 % idle) and the rows that fill
// a tile (7 % there) come on top.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "cluster_counts.h"
#include "zs_internal.h"

namespace {

#include "step_common.cuh"
#include "step_end.cuh"
#include "loss_common.cuh"
#include "mbar.cuh"
#include "tensor_core.cuh"
#include "elem.cuh"
#include "launch.cuh"

[[maybe_unused]] constexpr uint32_t kSiteHeadRow = 22, kSiteHeadSum = 23;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLowestFloat = -3.402823466e38f;

constexpr int64_t kTile = 256;  // rows, and entries of the vocabulary, that a block's sums cover
constexpr int64_t kMaxRows = 1 << 24, kMaxVocab = 1 << 24, kMaxWidth = 1 << 16;
constexpr int kMaxSplit = 16;               // parts of dH's sums
constexpr int64_t kPieceBytes = 1ll << 30;  // of a piece's gradient, where the caller leaves the choice

constexpr int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Rows between the statistics of two half tiles: not a power of 2, for the memory's channels.
__host__ __device__ constexpr int64_t part_pitch(int64_t rows_pad) { return rows_pad + 32; }

// ------------------------------------------------------------------ scratch ---

// What the rows kernel leaves for the others.
struct Counts {
    int32_t live;     // rows that are not left out
    float scale;      // d's power of 2
    float unscale;    // its inverse
    int32_t split;    // parts of dH's sums
};
// A live row.
struct __align__(16) Row {
    float top, log_sum;  // t, lnS
    float coef;          // c
    int32_t label;
};

// The parts of the scratch buffer, as offsets from its start.
struct Plan {
    int64_t rows_pad, tiles, piece, sums_room;
    int64_t index, slot, row, hidden, part, label_logit, d, total;
};
Plan plan_of(int64_t rows, int64_t width, int64_t vocab, int64_t piece, bool gradient) {
    Plan p = {};
    p.rows_pad = round_up(rows > 0 ? rows : 1, kTile);
    p.tiles = round_up(vocab, kTile) / kTile;
    int64_t at = 128;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += round_up(bytes, 128);
        return here;
    };
    p.index = take(4 * p.rows_pad);
    p.slot = take(4 * p.rows_pad);
    p.row = take((int64_t)sizeof(Row) * p.rows_pad);
    p.hidden = take(2 * p.rows_pad * width);
    if (gradient) {
        if (piece <= 0) piece = kPieceBytes / (2 * p.rows_pad);
        p.piece = piece < kTile ? kTile : piece > p.tiles * kTile ? p.tiles * kTile : round_up(piece, kTile);
        // fp32 sums of dH, several of them where there are few tiles
        const int64_t tiles = p.rows_pad / kTile * (round_up(width, kTile) / kTile);
        const int64_t parts = round_up(160, tiles) / tiles;
        p.sums_room = p.rows_pad * (parts < kMaxSplit ? parts : kMaxSplit);
        p.part = take(4 * p.sums_room * width);
        p.d = take(2 * p.rows_pad * p.piece);
    } else {
        p.part = take(2 * 8 * part_pitch(p.rows_pad) * p.tiles);
        p.label_logit = take(4 * p.rows_pad);
    }
    p.total = at;
    return p;
}
bool valid_sizes(int64_t rows, int64_t width, int64_t vocab) {
    return rows >= 0 && rows <= kMaxRows && vocab >= 1 && vocab <= kMaxVocab && width >= 8 && width <= kMaxWidth &&
           width % 8 == 0;
}
// The plan with the largest piece that fits; total = 0: none does.
Plan plan_within(int64_t rows, int64_t width, int64_t vocab, int64_t bytes) {
    Plan p = plan_of(rows, width, vocab, kTile, true);
    if (bytes < p.total) {
        p.total = 0;
        return p;
    }
    const int64_t more = (bytes - p.total) / (2 * p.rows_pad * kTile);
    return plan_of(rows, width, vocab, (more + 1) * kTile, true);
}

// ------------------------------------------------------------- live rows ---

struct HeadArgs {
    const void *hidden, *weight;
    int64_t rows, vocab, width, hidden_stride, weight_stride;
    float it;
    const int64_t* labels;
    const float *saved, *dlogp;  // gradient: else NULL
    const zs_ctrl* ctrl;
    float *logp, *saved_out;     // forward
    uint16_t* dhidden;
    int64_t dhidden_stride;
    uint16_t* dweight;
    int64_t dweight_stride;
    Counts* counts;
    int32_t *index, *slot;       // a live row's row; a row's place among the live ones, or -1
    Row* row;
    uint16_t* compact;           // [rows_pad][width]
    void* part;
    float* label_logit;
    uint16_t* d;                 // [rows_pad][piece]
    int64_t rows_pad, tiles, piece, sums_room;
    int32_t pairs;               // that make dH
};

constexpr int kStep = 64;  // k of a stage of the products' ring
__host__ __device__ constexpr int32_t tiles_of(int64_t n) { return (int32_t)((n + kTile - 1) / kTile); }
__host__ __device__ constexpr int32_t steps_of(int64_t n) { return (int32_t)((n + kStep - 1) / kStep); }

// The number of parts of dH's sums: with few tiles the CTA pairs would be idle.  The least
// cost, estimated in steps: rounds of tiles, each with a start and an end of some 12 steps,
// and what the parts cost to write and read.  A lane of the warp weighs a number.
__device__ int32_t split_of(const HeadArgs& a, int32_t live, int lane) {
    const int32_t m_tiles = tiles_of(live > 0 ? live : 1), tiles = m_tiles * tiles_of(a.width);
    const int32_t steps = steps_of(a.vocab < a.piece ? a.vocab : a.piece);  // (the same for every piece: the first one's)
    const int32_t room = (int32_t)(a.sums_room / (m_tiles * kTile)), s = lane + 1;
    float cost = 3.4e38f;
    if (s == 1 || (s <= kMaxSplit && s <= room && s * 8 <= steps))
        cost = (float)((tiles * s + a.pairs - 1) / a.pairs) * ((float)((steps + s - 1) / s) + 12.0f) +
               (s > 1 ? 0.3f * (float)(tiles * s) : 0.0f);
    float least = cost;
    for (int o = 16; o > 0; o >>= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
    return __ffs(__ballot_sync(0xffffffffu, cost == least));
}

constexpr int kRowThreads = 1024;
// Rows of one pass of the rows kernel's block; up to so many are numbered by every block of
// the gather kernel for itself instead, which saves a launch.
constexpr int kRowsEach = 8, kFewRows = 1024;

// Numbers live rows in their order, EACH to a thread, whose loads are under way together,
// and calls `emit` with a row, its number or -1, and what the products need of it.  Called by the
// whole block of THREADS; returns the number of live rows up to here.
template <int THREADS, int EACH, typename F>
__device__ int32_t number_rows(const HeadArgs& a, int64_t from, int32_t before, F emit) {
    constexpr int kWarps = THREADS / 32, kCounts = EACH * kWarps;
    const float factor = loss_scale_of(a.ctrl) * a.it;
    static_assert(kCounts % 32 == 0, "a warp scans the counts");
    __shared__ int32_t s_count[kCounts + 1];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int64_t label[EACH];
    float dlogp[EACH], top[EACH], log_sum[EACH];
    uint32_t votes[EACH];
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const int64_t i = from + k * THREADS + threadIdx.x;
        const bool grad = i < a.rows && a.dlogp != nullptr;
        label[k] = i < a.rows ? a.labels[i] : -1;
        dlogp[k] = grad ? a.dlogp[i] : 1.0f;
        top[k] = grad ? a.saved[2 * i] : 0.0f;
        log_sum[k] = grad ? a.saved[2 * i + 1] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        // (a row of nothing but -inf has no gradient, and perhaps an infinite hidden state)
        votes[k] = __ballot_sync(0xffffffffu, label[k] >= 0 && label[k] < a.vocab && dlogp[k] != 0.0f &&
                                                  log_sum[k] != -__int_as_float(0x7f800000));
        if (lane == 0) s_count[k * kWarps + warp] = __popc(votes[k]);
    }
    __syncthreads();
    if (warp == 0) {
        // counts become the numbers of live rows before them
        int32_t c[kCounts / 32], sum = 0;
#pragma unroll
        for (int q = 0; q < kCounts / 32; ++q) {
            c[q] = s_count[lane * (kCounts / 32) + q];
            sum += c[q];
        }
        int32_t scan = sum;
        for (int o = 1; o < 32; o *= 2) {
            const int32_t x = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += x;
        }
        int32_t n = before + scan - sum;
#pragma unroll
        for (int q = 0; q < kCounts / 32; ++q) {
            s_count[lane * (kCounts / 32) + q] = n;
            n += c[q];
        }
        if (lane == 31) s_count[kCounts] = n;
    }
    __syncthreads();
    const int32_t all = s_count[kCounts];
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const int64_t i = from + k * THREADS + threadIdx.x;
        if (i >= a.rows) break;
        const int32_t r = s_count[k * kWarps + warp] + __popc(votes[k] & ((1u << lane) - 1u));
        const float coef = a.dlogp == nullptr ? 0.0f : factor * dlogp[k];
        emit(i, votes[k] >> lane & 1u ? r : -1, Row{top[k], log_sum[k], coef, (int32_t)label[k]});
    }
    __syncthreads();
    return all;
}
// From the largest finite |c| of each thread: the numbers, and the power of 2 that takes it
// to [2^14, 2^15).  Called by the whole block of THREADS.
template <int THREADS>
__device__ void write_counts(const HeadArgs& a, int32_t live, float top) {
    __shared__ float s_top[THREADS / 32];
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (threadIdx.x % 32 == 0) s_top[threadIdx.x / 32] = top;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int32_t split = a.dlogp != nullptr ? split_of(a, live, threadIdx.x) : 1;
        for (int w = 0; w < THREADS / 32; ++w) top = fmaxf(top, s_top[w]);
        int e = top > 0.0f ? 14 - ilogbf(top) : 0;
        e = e > 120 ? 120 : e < -120 ? -120 : e;
        if (threadIdx.x == 0) *a.counts = Counts{live, scalbnf(1.0f, e), scalbnf(1.0f, -e), split};
    }
}
__device__ __forceinline__ float larger_finite(float top, float c) {
    return fabsf(c) <= 3.402823466e38f ? fmaxf(top, fabsf(c)) : top;
}

// Many rows: one block numbers them, since the numbers depend on all rows before.
__global__ void __launch_bounds__(kRowThreads) head_rows_kernel(const __grid_constant__ HeadArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    float top = 0.0f;
    int32_t live = 0;
    for (int64_t from = 0; from < a.rows; from += kRowsEach * kRowThreads)
        live = number_rows<kRowThreads, kRowsEach>(a, from, live, [&](int64_t i, int32_t r, const Row& row) {
            a.slot[i] = r;
            if (r < 0) return;
            top = larger_finite(top, row.coef);
            a.index[r] = (int32_t)i;
            a.row[r] = row;
        });
    write_counts<kRowThreads>(a, live, top);
}

// Copies the live rows' hidden states together, with zeros up to a whole tile, and
// writes the outputs of the rows that are left out: a warp to a row.  FEW: numbers the
// rows as well, in every block; the first one writes the numbers down.
template <bool FEW>
__global__ void __launch_bounds__(256) head_gather_kernel(const __grid_constant__ HeadArgs a) {
    __shared__ int32_t s_slot[FEW ? kFewRows : 1];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x % 32;
    const int32_t vectors = (int32_t)(a.width / 8);
    int32_t live;
    if (FEW) {
        float top = 0.0f;
        live = number_rows<256, kFewRows / 256>(a, 0, 0, [&](int64_t i, int32_t r, const Row& row) {
            s_slot[i] = r;
            if (r < 0 || blockIdx.x != 0) return;
            top = larger_finite(top, row.coef);
            a.index[r] = (int32_t)i;
            a.row[r] = row;
        });
        if (blockIdx.x == 0) write_counts<256>(a, live, top);
    } else {
        live = a.counts->live;
    }
    const int64_t fill = round_up(live, kTile) - live;
    for (int64_t i = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; i < a.rows + fill; i += (int64_t)gridDim.x * 8) {
        const int32_t slot = i >= a.rows ? (int32_t)(live + i - a.rows) : FEW ? s_slot[i] : a.slot[i];
        const bool copy = i < a.rows && slot >= 0;
        const uint4* from = reinterpret_cast<const uint4*>((const uint16_t*)a.hidden + i * a.hidden_stride);
        uint4* to = slot >= 0             ? reinterpret_cast<uint4*>(a.compact + (int64_t)slot * a.width)
                    : a.dhidden != nullptr ? reinterpret_cast<uint4*>(a.dhidden + i * a.dhidden_stride)
                                           : nullptr;
        if (to != nullptr && ZS_RANGE_OK(kSiteHeadRow, slot >= 0 ? slot : i, 1, slot >= 0 ? a.rows_pad : a.rows)) {
            for (int32_t k0 = lane; k0 < vectors; k0 += 4 * 32) {
                uint4 x[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) x[q] = copy && k0 + 32 * q < vectors ? from[k0 + 32 * q] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (k0 + 32 * q < vectors) to[k0 + 32 * q] = x[q];
            }
        }
        if (i >= a.rows) {
            if (lane == 0) a.row[slot] = Row{0.0f, 0.0f, 0.0f, -1};
        } else if (slot < 0) {
            if (lane == 0 && a.logp != nullptr) a.logp[i] = 0.0f;
            if (lane < 2 && a.saved_out != nullptr) a.saved_out[2 * i + lane] = 0.0f;
        }
    }
}

// ---------------------------------------------------------------- products ---

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fffffff); }
__device__ __forceinline__ float infinity() { return __int_as_float(0x7f800000); }

// The three products, each a 256 x 256 tile (of sums) at a time:
//   kLogits    H W^T: statistics of each row over the tile's entries
//   kGrad      the same over one piece of the vocabulary: d
//   kDHidden   d W over one piece
//   kDWeight   d^T H: the piece's rows of dW
//   kBack      both in one launch, since small calls wait for launches
enum { kLogits, kGrad, kDHidden, kDWeight, kBack };
constexpr bool of_logits(int mode) { return mode == kLogits || mode == kGrad; }

constexpr int kRowBytes = kStep * 2;                        // of an operand's row in a stage
constexpr int kBoxBytes = 64 * kRowBytes;                   // 64 m of 64 k, across k
constexpr int kBytesA = 128 * kRowBytes;                    // A's stage in a CTA
constexpr int columns_of(int ctas) { return (int)kTile / ctas; }  // of B in a CTA
constexpr int stage_bytes(int ctas) { return kBytesA + columns_of(ctas) * kRowBytes; }
constexpr int stages_of(int ctas) { return ctas == 2 ? 6 : 4; }
constexpr int kRing = 6 * stage_bytes(2);
static_assert(kRing == 4 * stage_bytes(1), "both fill the same shared memory");
constexpr int kMaxStages = 6;
// Steps that the tensor cores add up before their sums go to registers.  They cut a
// sum off at fp32's last place after every 16 k; over 4096 k that left logits off by
// 4e-6 of their size (a product in fp32 is off by 1e-7), over 512 k it leaves 5e-7.
constexpr int kRun = 8;
constexpr int kProductWarps = 8;                            // that take the sums
constexpr int kProductThreads = 128 + 32 * kProductWarps;
constexpr int kStaging = 4096;                              // bytes of a warp: 32 rows of 128
constexpr int kProductShared = kRing + kProductWarps * kStaging + 1024;
// Registers of a thread: 168 at launch (384 x 168 = 64,512); the copying and multiplying
// warps give up what the others take (128 x 72 + 256 x 216 = 64,512).
constexpr int kFewRegisters = 72, kManyRegisters = 216;
struct ProductArgs {
    HeadArgs h;
    int64_t first, count;  // the piece
    int32_t last;          // its end is the vocabulary's
};

// The tensor maps of a launch: A and B; else d and W for dH, d and H for dW.
struct Maps {
    CUtensorMap m[4];
};

// A product's tiles, and how many parts its sum is split into.
struct Tiles {
    int32_t m_tiles, n_tiles, split, steps;  // steps of kStep in the whole sum
    __device__ __forceinline__ int32_t units() const { return m_tiles * n_tiles * split; }
};
// Of a launch over the live rows: `back` is dW's, else empty.
struct Work2 {
    Tiles front, back;
};
template <int MODE, int CTAS>
__device__ __forceinline__ Work2 work_of(const ProductArgs& p, int32_t live) {
    Work2 w = {};
    if (of_logits(MODE)) w.front = Tiles{tiles_of(live), tiles_of(p.count), 1, steps_of(p.h.width)};
    if (MODE == kDHidden || MODE == kBack) w.front = Tiles{tiles_of(live), tiles_of(p.h.width), p.h.counts->split, steps_of(p.count)};
    if (MODE == kDWeight || MODE == kBack)
        w.back = Tiles{(int32_t)((p.count + CTAS * 128 - 1) / (CTAS * 128)), tiles_of(p.h.width), 1, steps_of(live)};
    return w;
}

// One tile, in the order in which they are taken.  Logits: groups of 16 tiles of rows go
// through the vocabulary together, so that a tile of W is read from memory once for each
// group and the group's rows stay in L2.  The others: tiles of the width run fastest (they
// share d), then rows.
struct Tile {
    int32_t m, n, part, from, to;  // from, to: steps
    bool weight;                   // of dW
};
template <int MODE>
__device__ __forceinline__ Tile tile_of(const Work2& both, int32_t u) {
    Tile t;
    t.weight = MODE == kDWeight || (MODE == kBack && u >= both.front.units());
    const Tiles& w = t.weight ? both.back : both.front;
    if (MODE == kBack && t.weight) u -= both.front.units();
    t.part = 0;
    t.from = 0;
    t.to = w.steps;
    if (of_logits(MODE)) {
        const int32_t group = 16 * w.n_tiles, g = u / group, first = g * 16, rest = u - g * group;
        const int32_t high = w.m_tiles - first < 16 ? w.m_tiles - first : 16;
        t.m = first + rest % high;
        t.n = rest / high;
    } else {
        t.n = u % w.n_tiles;
        const int32_t q = u / w.n_tiles;
        t.part = q / w.m_tiles;
        t.m = q - t.part * w.m_tiles;
        if (w.split > 1) {
            t.from = (int32_t)((int64_t)w.steps * t.part / w.split);
            t.to = (int32_t)((int64_t)w.steps * (t.part + 1) / w.split);
        }
    }
    return t;
}
// Columns of B in a tile: 128 where the width's last tile has no more.
template <int MODE>
__device__ __forceinline__ int32_t wide_of(const ProductArgs& p, int32_t n) {
    return !of_logits(MODE) && p.h.width - (int64_t)n * kTile <= 128 ? 128 : (int32_t)kTile;
}

struct Ring {
    uint64_t full[kMaxStages], empty[kMaxStages];  // full: the first CTA's counts both CTAs' copies
    uint64_t sums_full[2], sums_empty[2];          // sums_empty: the first CTA's counts both CTAs' warps
    uint64_t done;
    uint32_t sums;               // address of the tensor memory
    int32_t failed;              // a wait ran out
    int32_t issued;              // steps whose copies were issued,
    uint32_t bytes[kMaxStages];  // and what each CTA copied in the last ones
};

// The 128 columns of a thread's row, as 16-bit numbers or fp32, from registers to
// memory by way of the warp's staging place, so that a row's 128 bytes go out together.
// row_at(r): the place of row r of the warp's 32 in memory, NULL: nowhere; called by all
// lanes together.  Only the first `columns`.
template <int ELEM, typename R, typename F>
__device__ __forceinline__ void store_rows(uint8_t* staging, int lane, int32_t columns, R row_at, F vector_of) {
    constexpr int kEach = 16 / ELEM, kColumns = 128 / ELEM;  // of a vector; of 128 bytes
#pragma unroll
    for (int part = 0; part < 128 / kColumns; ++part) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint4*>(staging + lane * 128 + ((q ^ (lane & 7)) << 4)) = vector_of(part * kColumns + q * kEach);
        __syncwarp();
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int r = t * 4 + lane / 8, q = lane % 8;
            char* const to = row_at(r);
            const int32_t column = part * kColumns + q * kEach;
            if (to != nullptr && column < columns)
                *reinterpret_cast<uint4*>(to + column * ELEM) =
                    *reinterpret_cast<const uint4*>(staging + r * 128 + ((q ^ (r & 7)) << 4));
        }
        __syncwarp();
    }
}
// One of 32 values (a tree of selections: an index would put them into memory).
__device__ __forceinline__ float pick(const float* v, int32_t i) {
    float x[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = i & 16 ? v[k + 16] : v[k];
#pragma unroll
    for (int w = 8; w > 0; w /= 2)
#pragma unroll
        for (int k = 0; k < w; ++k) x[k] = i & w ? x[k + w] : x[k];
    return x[0];
}

// CTAS = 2: a pair of CTAs (a cluster of two) takes tile after tile.  In each CTA one
// thread copies its halves of A and B ahead into a ring of stages; one thread of the
// first CTA multiplies, 16 k at a time, into one of two sets of sums in tensor memory,
// kRun steps into each in turn; eight warps add the other set to sums in registers (a
// thread has half a row of the tile) and turn those into the tile's outputs.  CTAS = 1,
// for up to 128 rows: a CTA by itself has a tile of 128 rows, so that no half of the
// products is of rows that are not there.
template <typename T, int MODE, int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kProductThreads, 1)
    head_product_kernel(const __grid_constant__ Maps maps, const __grid_constant__ ProductArgs p) {
    constexpr int kStages = stages_of(CTAS), kStage = stage_bytes(CTAS);
    constexpr bool kAlongB = of_logits(MODE);  // B along k; A is too, but for dW
    extern __shared__ uint8_t s_raw[];
    __shared__ Ring ring;
    uint8_t* const stage0 = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    const int32_t pair = blockIdx.x / CTAS, pairs = gridDim.x / CTAS;
    const HeadArgs& a = p.h;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&ring.full[s], 1);
            mbar_init(&ring.empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&ring.sums_full[s], 1);
            mbar_init(&ring.sums_empty[s], CTAS * kProductWarps);
        }
        mbar_init(&ring.done, 1);
        ring.failed = 0;
        ring.issued = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int i = 0; i < 4; ++i) prefetch_map(&maps.m[i]);
    }
    if (warp == 2) tensor_alloc<CTAS>(&ring.sums);
    tensor_fence_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    tensor_fence_after();
    griddep_wait();
    const uint32_t sums = ring.sums;
    const int32_t live = a.counts->live;
    const Work2 w = work_of<MODE, CTAS>(p, live);
    const int32_t units = w.front.units() + w.back.units();

    if (warp < 4) give_registers<kFewRegisters>();
    if (warp == 0 && lane == 0) {
        // what earlier kernels wrote, seen by the copies
        asm volatile("fence.proxy.async.global;" ::: "memory");
        int32_t at = 0;
        bool ok = true;
        for (int32_t u = pair; u < units && ok; u += pairs) {
            const Tile t = tile_of<MODE>(w, u);
            const int32_t mine = wide_of<MODE>(p, t.n) / CTAS;  // columns of B in this CTA
            const uint32_t bytes = (uint32_t)(kBytesA + mine * kRowBytes);
            const CUtensorMap* const map_a = &maps.m[t.weight ? 2 : 0];
            const CUtensorMap* const map_b = &maps.m[t.weight ? 3 : 1];
            const int32_t m0 = t.m * (CTAS * 128) + (int32_t)rank * 128, n0 = t.n * (int32_t)kTile + (int32_t)rank * mine;
            for (int32_t k = t.from; k < t.to; ++k, ++at) {
                const int s = at % kStages;
                if (!mbar_wait<false, true>(&ring.empty[s], (uint32_t)(at / kStages + 1) & 1u, &ring.failed)) {
                    ok = false;
                    break;
                }
                ring.bytes[s] = bytes;
                ring.issued = at + 1;
                if (rank == 0) mbar_expect(&ring.full[s], CTAS * bytes);
                const uint32_t full = peer_addr(&ring.full[s], 0);
                uint8_t* const to_a = stage0 + s * kStage;
                uint8_t* const to_b = to_a + kBytesA;
                const int32_t x = k * kStep;
                if (!t.weight) {
                    copy_box<CTAS>(to_a, map_a, x, m0, full);
                } else {
                    copy_box<CTAS>(to_a, map_a, m0, x, full);
                    copy_box<CTAS>(to_a + kBoxBytes, map_a, m0 + 64, x, full);
                }
                if (kAlongB) {
                    copy_box<CTAS>(to_b, map_b, x, (int32_t)p.first + n0, full);
                } else {
                    const int32_t y = t.weight ? x : (int32_t)p.first + x;
                    for (int32_t c = 0; c < mine; c += 64) copy_box<CTAS>(to_b + c * kRowBytes, map_b, n0 + c, y, full);
                }
            }
        }
        // (the last products' arrivals at this CTA's barriers, before it leaves)
        for (int32_t i = at > kStages ? at - kStages : 0; i < at && ok; ++i)
            ok = mbar_wait<false, true>(&ring.empty[i % kStages], (uint32_t)(i / kStages) & 1u, &ring.failed);
    } else if (warp == 1 && lane == 0 && rank == 0) {
        int32_t at = 0, turn = 0;
        bool ok = true;
        for (int32_t u = pair; u < units && ok; u += pairs) {
            const Tile t = tile_of<MODE>(w, u);
            const uint32_t kind = product_kind<CTAS, T>((uint32_t)wide_of<MODE>(p, t.n), !t.weight, kAlongB);
            for (int32_t k = t.from; k < t.to; ++turn) {
                const int set = turn & 1;
                const int32_t stop = k + kRun < t.to ? k + kRun : t.to;
                ok = mbar_wait<false, true>(&ring.sums_empty[set], (uint32_t)(turn / 2 + 1) & 1u, &ring.failed);
                if (!ok) break;
                tensor_fence_after();
                for (bool add = false; k < stop; ++k, ++at, add = true) {
                    const int s = at % kStages;
                    ok = mbar_wait<false, true>(&ring.full[s], (uint32_t)(at / kStages) & 1u, &ring.failed);
                    if (!ok) break;
                    tensor_fence_after();
                    const uint8_t* const from = stage0 + s * kStage;
                    uint64_t da = operand(from, kBoxBytes, !t.weight), db = operand(from + kBytesA, kBoxBytes, kAlongB);
#pragma unroll
                    for (int q = 0; q < kStep / 16; ++q) {
                        multiply<CTAS>(sums + (uint32_t)set * 256u, da, db, kind, add || q > 0);
                        da += operand_step(!t.weight);
                        db += operand_step(kAlongB);
                    }
                    arrive_after_products<CTAS>(&ring.empty[s]);
                }
                if (!ok) break;
                arrive_after_products<CTAS>(&ring.sums_full[set]);
            }
        }
    } else if (warp >= 4) {
        take_registers<kManyRegisters>();
        const int quarter = warp % 4, side = (warp - 4) / 4;  // 32 rows, 128 columns
        uint8_t* const staging = stage0 + kRing + (warp - 4) * kStaging;
        const float k2 = a.it * kLog2e;
        bool ok = true;
        int32_t turn = 0;
        for (int32_t u = pair; u < units; u += pairs) {
            const Tile t = tile_of<MODE>(w, u);
            const bool mine = side == 0 || wide_of<MODE>(p, t.n) > 128;
            float v[128];
            // (a tile's first sums straight to their place, but dW's added to 0: with a few
            // rows, where its tiles are one step each, 155934 x 1104 took 143 us that way, 114 so)
            if (t.weight || t.from == t.to || !mine) {
#pragma unroll
                for (int i = 0; i < 128; ++i) v[i] = 0.0f;
            }
            for (int32_t k = t.from; k < t.to; k += kRun, ++turn) {
                const int set = turn & 1;
                ok = ok && all_lanes(mbar_wait<true, true>(&ring.sums_full[set], (uint32_t)(turn / 2) & 1u, &ring.failed));
                tensor_fence_after();
                const uint32_t from = sums + (uint32_t)(set * 256 + side * 128) + ((uint32_t)quarter * 32u << 16);
                if (!t.weight && mine && ok && k == t.from) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) tensor_load(from + (uint32_t)c * 32u, v + c * 32);
                    tensor_load_wait();
#pragma unroll
                    for (int c = 0; c < 4; ++c) loaded(v + c * 32);
                } else if (mine && ok) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float x[32];
                        tensor_load(from + (uint32_t)c * 32u, x);
                        tensor_load_wait();
                        loaded(x);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[c * 32 + i] += x[i];
                    }
                }
                tensor_fence_before();
                __syncwarp();
                // (not after a wait that ran out: an arrival out of turn could stand for another
                // warp's, and its sums would be written over unread)
                if (ok && lane == 0) arrive_at(peer_addr(&ring.sums_empty[set], 0));
            }
            if (!ok) {
#pragma unroll
                for (int i = 0; i < 128; ++i) v[i] = quiet_nan();
            }
            if (!mine) continue;
            const int64_t r0 = (int64_t)t.m * (CTAS * 128) + rank * 128 + quarter * 32, r = r0 + lane;  // the thread's row of the tile,
            const int64_t j0 = (int64_t)t.n * kTile + side * 128;                        // and its first column
            if (MODE == kLogits) {
                const int32_t label = a.row[r].label - (int32_t)j0;
                if (__any_sync(0xffffffffu, (uint32_t)label < 128u)) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float x = pick(v + c * 32, label & 31);
                        if (label >> 5 == c) a.label_logit[r] = x;
                    }
                }
                if (j0 + 128 > p.count) {
#pragma unroll
                    for (int i = 0; i < 128; ++i) v[i] = j0 + i < p.count ? v[i] : -infinity();
                }
                float high[4] = {kLowestFloat, kLowestFloat, kLowestFloat, kLowestFloat}, add[4] = {};
#pragma unroll
                for (int i = 0; i < 128; ++i) high[i % 4] = fmaxf(high[i % 4], v[i]);
                const float top = fmaxf(fmaxf(high[0], high[1]), fmaxf(high[2], high[3]));
#pragma unroll
                for (int i = 0; i < 128; ++i) add[i % 4] += exp2_approx((v[i] - top) * k2);
                ((float2*)a.part)[(2 * (int64_t)t.n + side) * part_pitch(a.rows_pad) + r] =
                    make_float2(top, (add[0] + add[1]) + (add[2] + add[3]));
            } else if (MODE == kGrad) {
                const Row row = a.row[r];
                const float shift = row.log_sum * kLog2e, coef = row.coef * a.counts->scale;
                const int32_t label = row.label - (int32_t)(p.first + j0);
#pragma unroll
                for (int i = 0; i < 128; ++i) v[i] = -coef * exp2_approx(fmaf(v[i] - row.top, k2, -shift));
                if (__any_sync(0xffffffffu, (uint32_t)label < 128u)) {
#pragma unroll
                    for (int i = 0; i < 128; ++i) v[i] += label == i ? coef : 0.0f;
                }
                if (j0 + 128 > p.count) {
#pragma unroll
                    for (int i = 0; i < 128; ++i) v[i] = j0 + i < p.count ? v[i] : 0.0f;
                }
                // (rows that only fill the tile are 0, whatever W holds)
                const bool none = coef == 0.0f;
                const bool in = ZS_RANGE_OK(kSiteHeadSum, r0, 32, a.rows_pad) && ZS_RANGE_OK(kSiteHeadSum, j0, 128, a.piece);
                char* const to = reinterpret_cast<char*>(a.d + r0 * a.piece + j0);
                store_rows<2>(staging, lane, in ? 128 : 0, [&](int i) { return to + i * a.piece * 2; }, [&](int j) {
                    return none ? make_uint4(0, 0, 0, 0)
                                : make_uint4(narrow2<T>(v[j], v[j + 1]), narrow2<T>(v[j + 2], v[j + 3]),
                                             narrow2<T>(v[j + 4], v[j + 5]), narrow2<T>(v[j + 6], v[j + 7]));
                });
            } else {
                const int64_t left = a.width - j0;
                const int32_t columns = left < 128 ? (int32_t)left : 128;
                if (!t.weight && !(w.front.split == 1 && p.first == 0 && p.last)) {
                    // (rows that only fill the tile have room as well)
                    const int64_t at = (int64_t)t.part * w.front.m_tiles * kTile + r0;
                    const bool in = ZS_RANGE_OK(kSiteHeadSum, at, 32, a.sums_room);
                    float* const to = (float*)a.part + at * a.width + j0;
                    if (p.first > 0 && in) {
                        const float* const row = to + lane * a.width;
#pragma unroll
                        for (int i = 0; i < 128; i += 4) {
                            if (i >= columns) break;
                            const float4 x = *reinterpret_cast<const float4*>(row + i);
                            v[i] += x.x, v[i + 1] += x.y, v[i + 2] += x.z, v[i + 3] += x.w;
                        }
                    }
                    __syncwarp();
                    store_rows<4>(staging, lane, in ? columns : 0, [&](int i) { return reinterpret_cast<char*>(to + i * a.width); }, [&](int j) {
                        return make_uint4(__float_as_uint(v[j]), __float_as_uint(v[j + 1]), __float_as_uint(v[j + 2]),
                                          __float_as_uint(v[j + 3]));
                    });
                } else {
                    const float unscale = a.counts->unscale;
                    // the lane's row of dH lies anywhere, a row of dW after the one before
                    uint16_t* row = nullptr;
                    if (!t.weight && r < live && ZS_RANGE_OK(kSiteHeadRow, a.index[r], 1, a.rows))
                        row = a.dhidden + a.index[r] * a.dhidden_stride + j0;
                    uint16_t* const to = a.dweight + (p.first + r0) * a.dweight_stride + j0;
                    const int32_t rows = (int32_t)(p.count - r0 < 32 ? p.count - r0 : 32);
                    const bool in = !t.weight || rows < 1 || ZS_RANGE_OK(kSiteHeadRow, p.first + r0, rows, a.vocab);
                    auto row_at = [&](int i) {
                        if (!t.weight)
                            return reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), i));
                        return i < rows ? reinterpret_cast<char*>(to + i * a.dweight_stride) : nullptr;
                    };
                    store_rows<2>(staging, lane, in ? columns : 0, row_at, [&](int j) {
                        uint32_t x[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[i] = narrow2<T>(v[j + 2 * i] * unscale, v[j + 2 * i + 1] * unscale);
                        return make_uint4(x[0], x[1], x[2], x[3]);
                    });
                }
            }
        }
    }
    __syncwarp();
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    // Where a wait ran out, products and copies may be under way: neither CTA leaves
    // before the products are done and the barriers of the last steps that either
    // issued have counted their copies (of a step that one of the two did not reach,
    // that one's are made up for).
    if ((load_from_peer(&ring.failed, 0) | load_from_peer(&ring.failed, CTAS - 1)) != 0 && rank == 0 && threadIdx.x == 32) {
        signal_after_products<CTAS>(&ring.done);
        drain(&ring.done, 0);
        const int32_t mine = ring.issued, other = load_from_peer(&ring.issued, CTAS - 1);
        const int32_t most = mine > other ? mine : other;
        for (int32_t i = most > kStages ? most - kStages : 0; i < most; ++i) {
            const int s = i % kStages;
            if (i >= mine) mbar_expect(&ring.full[s], (uint32_t)load_from_peer((const int32_t*)&ring.bytes[s], CTAS - 1));
            if (i >= other) mbar_give(&ring.full[s], ring.bytes[s]);
            drain(&ring.full[s], (uint32_t)(i / kStages) & 1u);
        }
    }
    __syncwarp();
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    tensor_fence_after();
    if (warp == 2) tensor_free<CTAS>(sums);
}

// Joins the statistics of the rows' half tiles: 32 rows to a block, 16 threads to a row.
__global__ void __launch_bounds__(512) head_join_kernel(const __grid_constant__ HeadArgs a) {
    __shared__ float2 s_part[16][32];
    const int lane = threadIdx.x % 32, group = threadIdx.x / 32;
    const int64_t r = (int64_t)blockIdx.x * 32 + lane;
    griddep_wait();
    const int32_t live = a.counts->live;
    if ((int64_t)blockIdx.x * 32 >= live) return;
    const float k = a.it * kLog2e;
    float top = kLowestFloat, s = 0.0f;
    auto join = [&](float2 q) {
        const float high = fmaxf(top, q.x);
        s = s * exp2_approx((top - high) * k) + q.y * exp2_approx((q.x - high) * k);
        top = high;
    };
    const float2* part = (const float2*)a.part + r;  // (rows up to a whole tile have statistics)
    const int64_t pitch = part_pitch(a.rows_pad);
    const int32_t n = (int32_t)(2 * a.tiles);
    for (int32_t t = group; t < n; t += 8 * 16) {
        float2 q[8];
        // (all eight loads under way at once: past the end the last one's again)
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = part[(t + 16 * i < n ? t + 16 * i : n - 1) * pitch];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (t + 16 * i < n) join(q[i]);
    }
    s_part[group][lane] = make_float2(top, s);
    __syncthreads();
    if (group != 0 || r >= live) return;
    for (int g = 1; g < 16; ++g) join(s_part[g][lane]);
    const int64_t i = a.index[r];
    const float log_sum = logf(s);
    a.logp[i] = s == 0.0f ? log_sum : (a.label_logit[r] - top) * a.it - log_sum;
    if (a.saved_out != nullptr) {
        a.saved_out[2 * i] = top;
        a.saved_out[2 * i + 1] = log_sum;
    }
}

// Joins the parts of dH's sums: a warp to 128 columns of a row.
template <typename T>
__global__ void __launch_bounds__(256) head_dhidden_kernel(const __grid_constant__ ProductArgs p) {
    griddep_wait();
    const HeadArgs& a = p.h;
    const int32_t live = a.counts->live, split = a.counts->split;
    if (split == 1 && p.first == 0) return;  // (one piece: the product wrote dH)
    const int lane = threadIdx.x % 32;
    const float unscale = a.counts->unscale;
    const int64_t part = (int64_t)tiles_of(live) * kTile * a.width;
    const int32_t each = (int32_t)((a.width + 127) / 128);
    for (int64_t u = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; u < (int64_t)live * each; u += (int64_t)gridDim.x * 8) {
        const int64_t r = u / each, k = (u - r * each) * 128 + lane * 4;
        if (k >= a.width) continue;
        const float* from = (const float*)a.part + r * a.width + k;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int32_t q = 0; q < split; q += 4) {
            float4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(from + (q + i < split ? q + i : split - 1) * part);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (q + i < split) s = make_float4(s.x + x[i].x, s.y + x[i].y, s.z + x[i].z, s.w + x[i].w);
        }
        *reinterpret_cast<uint2*>(a.dhidden + (int64_t)a.index[r] * a.dhidden_stride + k) =
            make_uint2(narrow2<T>(s.x * unscale, s.y * unscale), narrow2<T>(s.z * unscale, s.w * unscale));
    }
}

// ------------------------------------------------------------------- launches ---

// The tensor map of a matrix of 16-bit elements, `wide` of them to a row: boxes of 64
// elements (a row of the swizzle) by `box_rows` rows.  Outside the matrix are zeros.
int32_t make_map(CUtensorMap* map, int32_t type, const void* base, int64_t rows, int64_t wide, int64_t stride,
                 uint32_t box_rows) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return (Encode)f;
    }();
    if (encode == nullptr) return zs::fail_with(ZS_ERR_CUDA, "cuTensorMapEncodeTiled: not found in the driver");
    const cuuint64_t dims[2] = {(cuuint64_t)wide, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {64, box_rows}, one[2] = {1, 1};
    const CUresult rc = encode(map, type == ZS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                               const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return rc == CUDA_SUCCESS ? ZS_OK : zs::fail_with(ZS_ERR_CUDA, "cuTensorMapEncodeTiled: refused a matrix of the head");
}

// Pairs of CTAs (CTAS = 1: CTAs) that run at once; 0: a CUDA error, recorded.
template <typename T, int MODE, int CTAS>
int pairs_of() {
    return clusters_of((const void*)head_product_kernel<T, MODE, CTAS>, kProductThreads, CTAS, kProductShared);
}
template <typename T, int MODE, int CTAS>
int32_t launch_product(const ProductArgs& p, const Maps& maps, int pairs, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(CTAS * pairs));
    cfg.blockDim = dim3(kProductThreads);
    cfg.dynamicSmemBytes = kProductShared;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, head_product_kernel<T, MODE, CTAS>, maps, p);
    if (err != cudaSuccess) return zs::cuda_fail(err, "head_product_kernel");
    return zs::check_launch("head_product_kernel");
}

bool valid_stride(int64_t rows, int64_t width, int64_t stride) {
    return rows <= 1 || (stride >= width && stride <= 1ll << 38);  // (tensor maps: bytes below 2^40)
}

int32_t check_head(const zs_head* h) {
    if (h == nullptr || !valid_sizes(h->rows, h->width, h->vocab) || (h->type != ZS_F16 && h->type != ZS_BF16) ||
        h->reserved != 0 || !(h->inv_temperature >= 1e-6 && h->inv_temperature <= 1e6))
        return ZS_ERR_ARG;
    if (h->weight == nullptr || (h->rows > 0 && h->hidden == nullptr)) return ZS_ERR_ARG;
    if (!valid_stride(h->rows, h->width, h->hidden_stride) || !valid_stride(h->vocab, h->width, h->weight_stride))
        return ZS_ERR_ARG;
    if (!zs::aligned_to(h->hidden, 16) || !zs::aligned_to(h->weight, 16) || (h->rows > 1 && h->hidden_stride % 8 != 0) ||
        (h->vocab > 1 && h->weight_stride % 8 != 0))
        return ZS_ERR_ALIGN;
    return ZS_OK;
}

HeadArgs args_of(const zs_head* h, const Plan& p, void* work) {
    HeadArgs a = {};
    char* base = (char*)work;
    a.hidden = h->hidden;
    a.weight = h->weight;
    a.rows = h->rows;
    a.vocab = h->vocab;
    a.width = h->width;
    a.hidden_stride = h->rows > 1 ? h->hidden_stride : h->width;
    a.weight_stride = h->vocab > 1 ? h->weight_stride : h->width;
    a.it = (float)h->inv_temperature;
    a.counts = (Counts*)base;
    a.index = (int32_t*)(base + p.index);
    a.slot = (int32_t*)(base + p.slot);
    a.row = (Row*)(base + p.row);
    a.compact = (uint16_t*)(base + p.hidden);
    a.part = base + p.part;
    a.label_logit = (float*)(base + p.label_logit);
    a.d = (uint16_t*)(base + p.d);
    a.rows_pad = p.rows_pad;
    a.tiles = p.tiles;
    a.piece = p.piece;
    a.sums_room = p.sums_room;
    return a;
}

int32_t launch_rows(const HeadArgs& a, cudaStream_t stream) {
    const int64_t most = 6 * zs::device_sm_count(), blocks = (a.rows + kTile + 7) / 8;
    const dim3 grid((unsigned)(blocks < most ? blocks : most));
    if (a.rows <= kFewRows) return launch(head_gather_kernel<true>, grid, 256, stream, "head_gather_kernel", a);
    ZS_TRY(launch(head_rows_kernel, dim3(1), kRowThreads, stream, "head_rows_kernel", a));
    return launch(head_gather_kernel<false>, grid, 256, stream, "head_gather_kernel", a);
}

template <typename T> constexpr int32_t type_of();
template <> constexpr int32_t type_of<__half>() { return ZS_F16; }
template <> constexpr int32_t type_of<__nv_bfloat16>() { return ZS_BF16; }

template <typename T, int CTAS>
int32_t launch_logp(const HeadArgs& a, cudaStream_t stream) {
    Maps maps;
    ZS_TRY(make_map(&maps.m[0], type_of<T>(), a.compact, a.rows_pad, a.width, a.width, 128));
    ZS_TRY(make_map(&maps.m[1], type_of<T>(), a.weight, a.vocab, a.width, a.weight_stride, columns_of(CTAS)));
    maps.m[2] = maps.m[3] = maps.m[1];
    const int pairs = pairs_of<T, kLogits, CTAS>();
    if (pairs < 1) return ZS_ERR_CUDA;
    ZS_TRY(launch_rows(a, stream));
    ZS_TRY((launch_product<T, kLogits, CTAS>(ProductArgs{a, 0, a.vocab, 1}, maps, pairs, stream)));
    return launch(head_join_kernel, dim3((unsigned)(round_up(a.rows, 32) / 32)), 512, stream, "head_join_kernel", a);
}

template <typename T, int CTAS>
int32_t launch_grad(HeadArgs a, cudaStream_t stream) {
    // the operands: H and W along k; d along k and W across, d and H across
    Maps logits, back;
    ZS_TRY(make_map(&logits.m[0], type_of<T>(), a.compact, a.rows_pad, a.width, a.width, 128));
    ZS_TRY(make_map(&logits.m[1], type_of<T>(), a.weight, a.vocab, a.width, a.weight_stride, columns_of(CTAS)));
    logits.m[2] = logits.m[3] = logits.m[1];
    ZS_TRY(make_map(&back.m[0], type_of<T>(), a.d, a.rows_pad, a.piece, a.piece, 128));
    ZS_TRY(make_map(&back.m[1], type_of<T>(), a.weight, a.vocab, a.width, a.weight_stride, 64));
    ZS_TRY(make_map(&back.m[2], type_of<T>(), a.d, a.rows_pad, a.piece, a.piece, 64));
    ZS_TRY(make_map(&back.m[3], type_of<T>(), a.compact, a.rows_pad, a.width, a.width, 64));
    const int pairs = pairs_of<T, kGrad, CTAS>();
    // dH and dW in one launch where that takes some 100 us (4728 x 4116 x 1104 117 us for 135).
    // With longer ones the tiles, dealt in turn, come out less even, and a kernel that
    // looks at each tile's kind is slower (2048 x 50257 x 1600 580 us for 568, 7 x 155934 x 1104, of
    // 256 rows in tiles, 349 for 304).
    const bool together = a.dhidden != nullptr && a.dweight != nullptr &&
                          6.0 * (double)a.rows_pad * (double)a.vocab * (double)a.width < 2e11;
    a.pairs = together ? pairs_of<T, kBack, CTAS>() : pairs_of<T, kDHidden, CTAS>();
    const int pairs_w = pairs_of<T, kDWeight, 2>();
    if (pairs < 1 || a.pairs < 1 || pairs_w < 1) return ZS_ERR_CUDA;
    ZS_TRY(launch_rows(a, stream));
    ProductArgs p = {a, 0, 0, 0};
    for (p.first = 0;; p.first += a.piece) {
        p.last = p.first + a.piece >= a.vocab;
        p.count = p.last ? a.vocab - p.first : a.piece;
        ZS_TRY((launch_product<T, kGrad, CTAS>(p, logits, pairs, stream)));
        if (together) {
            ZS_TRY((launch_product<T, kBack, CTAS>(p, back, a.pairs, stream)));
        } else {
            if (a.dhidden != nullptr) ZS_TRY((launch_product<T, kDHidden, CTAS>(p, back, a.pairs, stream)));
            if (a.dweight != nullptr) ZS_TRY((launch_product<T, kDWeight, 2>(p, back, pairs_w, stream)));
        }
        if (p.last) break;
    }
    if (a.dhidden == nullptr) return ZS_OK;
    const int64_t most = 8 * zs::device_sm_count(), blocks = a.rows * ((a.width + 127) / 128) / 8 + 1;
    return launch(head_dhidden_kernel<T>, dim3((unsigned)(blocks < most ? blocks : most)), 256, stream, "head_dhidden_kernel", p);
}

// Calls f with a value of the type, and the CTAs of a tile as a constant: one for up to
// 128 rows (4 x 32000 x 4096: 56.6 us for 63.9), two above.
template <typename F>
int32_t with_head(const zs_head* h, F f) {
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    if (h->type == ZS_F16) return h->rows <= 128 ? f(__half(), one) : f(__half(), two);
    return h->rows <= 128 ? f(__nv_bfloat16(), one) : f(__nv_bfloat16(), two);
}

}  // namespace

namespace zs {
uint64_t take_fault_head() { return take_fault(); }
int32_t set_wait_limit_head(int32_t tries) { return set_unit_wait_limit(tries); }
}  // namespace zs

extern "C" {

ZS_API int64_t zero_head_work_bytes(int64_t rows, int64_t width, int64_t vocab, int64_t piece, int32_t gradient) {
    if (!valid_sizes(rows, width, vocab) || piece < 0 || (gradient != 0 && gradient != 1)) return ZS_ERR_ARG;
    return plan_of(rows, width, vocab, piece, gradient == 1).total;
}

ZS_API int32_t zero_head_logp_async(const zs_head* h, const int64_t* labels, float* logp, float* saved,
                                    void* work_dev, int64_t work_bytes, void* stream) {
    zs::NvtxRange nvtx_range("zero_head_logp_async");
    ZS_TRY(check_head(h));
    if (h->rows == 0) return ZS_OK;
    if (labels == nullptr || logp == nullptr || work_dev == nullptr) return ZS_ERR_ARG;
    if (!zs::aligned_to(labels, 8) || !zs::aligned_to(logp, 4) || !zs::aligned_to(saved, 4) || !zs::aligned_to(work_dev, 128))
        return ZS_ERR_ALIGN;
    const Plan p = plan_of(h->rows, h->width, h->vocab, 0, false);
    if (work_bytes < p.total) return ZS_ERR_ARG;
    HeadArgs a = args_of(h, p, work_dev);
    a.labels = labels;
    a.logp = logp;
    a.saved_out = saved;
    return with_head(h, [&](auto t, auto ctas) { return launch_logp<decltype(t), decltype(ctas)::value>(a, (cudaStream_t)stream); });
}

ZS_API int32_t zero_head_logp_grad_async(const zs_head* h, const int64_t* labels, const float* saved,
                                         const float* dlogp, const zs_ctrl* ctrl_dev, void* dhidden,
                                         int64_t dhidden_stride, void* dweight, int64_t dweight_stride,
                                         void* work_dev, int64_t work_bytes, void* stream) {
    zs::NvtxRange nvtx_range("zero_head_logp_grad_async");
    ZS_TRY(check_head(h));
    if (work_dev == nullptr || (dhidden == nullptr && dweight == nullptr)) return ZS_ERR_ARG;
    if (h->rows > 0 && (labels == nullptr || saved == nullptr || dlogp == nullptr)) return ZS_ERR_ARG;
    if ((dhidden != nullptr && !valid_stride(h->rows, h->width, dhidden_stride)) ||
        (dweight != nullptr && !valid_stride(h->vocab, h->width, dweight_stride)))
        return ZS_ERR_ARG;
    if (!zs::aligned_to(labels, 8) || !zs::aligned_to(saved, 4) || !zs::aligned_to(dlogp, 4) || !zs::aligned_to(ctrl_dev, 8) ||
        !zs::aligned_to(dhidden, 16) || !zs::aligned_to(dweight, 16) || !zs::aligned_to(work_dev, 128) ||
        (dhidden != nullptr && h->rows > 1 && dhidden_stride % 8 != 0) ||
        (dweight != nullptr && h->vocab > 1 && dweight_stride % 8 != 0))
        return ZS_ERR_ALIGN;
    const Plan p = plan_within(h->rows, h->width, h->vocab, work_bytes);
    if (p.total == 0) return ZS_ERR_ARG;
    if (h->rows == 0 && dweight == nullptr) return ZS_OK;
    HeadArgs a = args_of(h, p, work_dev);
    a.labels = labels;
    a.saved = saved;
    a.dlogp = dlogp;
    a.ctrl = ctrl_dev;
    a.dhidden = (uint16_t*)dhidden;
    a.dhidden_stride = h->rows > 1 ? dhidden_stride : h->width;
    a.dweight = (uint16_t*)dweight;
    a.dweight_stride = h->vocab > 1 ? dweight_stride : h->width;
    return with_head(h, [&](auto t, auto ctas) { return launch_grad<decltype(t), decltype(ctas)::value>(a, (cudaStream_t)stream); });
}

}  // extern "C"
