// The adapters' products on the tensor cores (bf16): three kernels make up both passes.
//
//   products : P[m, r] = sum_c U[m, c] T_a[c, r]             H = X A^T (forward), G = s dY B (backward)
//   update   : out[m, c] = in[m, c] + sum_r P[m, r] T_a[c, r]    out = Y + s H B^T,   dX + G A
//   columns  : D_a[c, r] = sum_m U[m, c] P[m, r]             dA = G^T X,        dB = dY^T (s H)
//
// Each streams its [rows, columns] matrix once and does 2 R (4 R where P is split) flops for each element: at
// ranks up to 32 far below what the tensor cores sustain beside a full HBM stream, so these kernels are
// built as streams: cp.async rings, 16-byte vectors, rows gathered through the plan by their own pointers. What
// multiplies follows from what the result needs. G, dA and dB take tcgen05 out of the ring as it lies, with the sums in
// tensor memory: one thread issues a stage, and the other warps only load. H is handed out in float32, which tensor
// memory's truncating sums over thousands of columns would cost digits, and `update` starts from `in` and
// writes each element once: these two keep mma.sync and sums in registers.
//
// Ranks are padded to 16, 32, 64 or 128 (RT). Whole passes, us as graph replays beside what their bytes take at the measured
// 6.55 TB/s. Forward, 4096 x 4096 x 14336, rank 16, eight adapters: 58 (41.7); 16384 x 4096 x 4096: 85 (61.8). Backward, one
// adapter of 4096 x 4096 x 4096, rank 16: 39.3 (20.6), rank 64: 57, rank 128: 98; four of 8192 x 768 x 2304, rank 32: 47 (11.9).
//
// P between the kernels: rows in plan order, [2][RT] bf16 each: the value rounded to bf16, and
// what that left out, rounded again (2^-17 of the value is lost). The products with both parts are
// added in float32. One bf16 part alone would add an error as large as the output's own rounding.
#include "ss1_adapter.cuh"
#include "ptx_sm100.cuh"

namespace ss1 {
namespace ada {
namespace {

using namespace op;
using bf16 = __nv_bfloat16;

constexpr int kThreads = 256, kPortableCluster = 8;

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
// d += a b: 16 x 8 float32, a 16 x 16 (rows g, g + 8 of lane / 4), b 16 x 8.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16-byte asynchronous copy; zeros where `ok` is false (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

// The two bf16 parts of a pair of values. A value without a finite first part has no second one.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
    const bf16 hx = __float2bfloat16_rn(x), hy = __float2bfloat16_rn(y);
    const float fx = __bfloat162float(hx), fy = __bfloat162float(hy);
    const __nv_bfloat162 h = __halves2bfloat162(hx, hy);
    const __nv_bfloat162 l = __floats2bfloat162_rn(fabsf(fx) < INFINITY ? x - fx : 0.0f, fabsf(fy) < INFINITY ? y - fy : 0.0f);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
}

// Instruction descriptor for operands whose contiguous side is M (A) or N (B): bits 15 and 16.
__host__ __device__ constexpr uint32_t idesc_mn(int N, bool a_mn, bool b_mn) {
    return ptx::idesc_bf16_f32(128, N) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
}
// A swizzled [rows][64] box in shared memory, 128 bytes a row, as an operand with the rows along the reduction: 8 rows are
// one 1024-byte atom, `next` bytes lead to the box of the next 64 elements.
__device__ __forceinline__ uint64_t desc_mn(uint32_t at, uint32_t next) { return ptx::smem_desc(at, next, 1024, ptx::kLayoutSW128); }
// The same kind of box with the rows along M or N.
__device__ __forceinline__ uint64_t desc_k(uint32_t at) { return ptx::smem_desc(at, 16, 1024, ptx::kLayoutSW128); }

// How waits are bounded: two seconds, where the products of a stage take a microsecond. A test's kernels (others, so
// that these pay nothing for it: 2 %) take a Watch in its place.
struct Unwatched {
    static constexpr uint64_t limit_ns = 2000000000ull;
    static constexpr int withhold = 0;
};

// The tensor core's part of a CTA: one completion barrier a ring slot, and what says that a wait gave up. Then no wait of the
// CTA lasts any more, its results are NaN, the status word is set, and a last commit sees to it that whatever was issued
// ends before its memory is freed (or a second limit passes). The loops issue as before: a test there of whether to go on cost
// 2 % (4096 x 4096 x 14336: 67.5 -> 68.8 us).
constexpr int kSlots = 6;
__device__ int32_t g_status;      // the first time-out since it was read: kernel id << 8 | 0x80 | site
struct TensorState {
    uint64_t done[kSlots];        // the last one: for the end after a wait gave up
    uint32_t tmem;
    int gave_up, never;           // never: 0
};
__device__ __forceinline__ void tensor_begin(TensorState& t, uint32_t columns) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) ptx::mbar_init(&t.done[i], 1);
        t.gave_up = t.never = 0;
        ptx::fence_mbar_init();
    }
    if (threadIdx.x < 32) {
        ptx::tmem_alloc(&t.tmem, columns);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
}
__device__ __forceinline__ bool tensor_fine(const TensorState& t) { return *(const volatile int*)&t.gave_up == 0; }
template <typename W>
__device__ __forceinline__ void tensor_wait(TensorState& t, int slot, uint32_t parity, const W& watch) {
    if (!ptx::mbar_wait(&t.done[slot], parity, &t.gave_up, watch.limit_ns)) *(volatile int*)&t.gave_up = 1;
}
// One thread; out of line, since small calls wait for their code to be fetched.
__device__ __noinline__ void tensor_gave_up(TensorState* t, uint64_t limit_ns, int site) {
    atomicCAS(&g_status, 0, (kStatusKernelAdapter << 8) | 0x80 | site);
    ptx::umma_commit(&t->done[kSlots - 1]);
    ptx::mbar_wait(&t->done[kSlots - 1], 0, &t->never, limit_ns);
}
// All threads, after the last wait and the last read of tensor memory.
template <typename W>
__device__ __forceinline__ void tensor_end(TensorState& t, uint32_t columns, const W& watch, int site) {
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (!tensor_fine(t)) {
        if (threadIdx.x == 0) tensor_gave_up(&t, watch.limit_ns, site);
        __syncthreads();
    }
    if (threadIdx.x < 32) ptx::tmem_dealloc(t.tmem, columns);
}

struct Tile {
    int adapter, first, rows;   // adapter -1: rows without one
};
__device__ __forceinline__ Tile tile_of(const PlanView& plan, int i, int M) {
    if (plan.rows == nullptr) return Tile{0, i * kTile, min(kTile, M - i * kTile)};
    const int4 t = plan.tiles[i];
    return Tile{t.x, t.y, t.y < 0 ? 0 : min(t.z, min(kTile, M - t.y))};   // a plan of another batch leads to no other places
}
// The batch row at a place of the plan, -1 if there is none.
__device__ __forceinline__ int row_at(const PlanView& plan, int place, int M) {
    const int m = plan.rows == nullptr ? place : plan.rows[place];
    return (unsigned)m < (unsigned)M ? m : -1;
}

// The forward's first kernel starts while the plan is still being made (by one CTA, in 6 us) and brings X, then Y,
// into L2 meanwhile: whatever wrote them is over, since the plan's kernel has waited for it. 4096 x 4096 x 14336 (X 33 MB,
// Y 117 MB), rank 16, eight adapters: 63.5 us without, 62.2 with 33 MB, 60.8 with 48 and 59.6 with 80; 4096 x 4096 x
// 4096: 29.6 without, 26.8 with. The backward, whose first kernel waits longer for less, has nothing of it (1 % either way).
constexpr int64_t kAhead = 80ll << 20;
struct Ahead {
    const void* at[2];
    int64_t bytes[2];      // whole 16 bytes
};
Ahead ahead_of(const Call& c, const void* X, const void* Y) {
    Ahead h = {};
    if (!c.planned) return h;
    h.at[0] = X;
    h.at[1] = Y;
    h.bytes[0] = c.M * c.K * 2 < kAhead ? c.M * c.K * 2 : kAhead;
    h.bytes[1] = c.M * c.N * 2 < kAhead - h.bytes[0] ? c.M * c.N * 2 : kAhead - h.bytes[0];
    return h;
}
__device__ __forceinline__ void bring_ahead(const Ahead& h, int cta, int ctas) {
    if (threadIdx.x != 0) return;
    constexpr int64_t kPiece = 16384;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        for (int64_t i = (int64_t)cta * kPiece; i < h.bytes[k]; i += (int64_t)ctas * kPiece) {
            const uint32_t size = (uint32_t)(h.bytes[k] - i < kPiece ? h.bytes[k] - i : kPiece);
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"((const char*)h.at[k] + i), "r"(size) : "memory");
        }
}

// ---- prepare ---------------------------------------------------------------------------------

// What the other kernels read in another form, in one launch: CTAs 0 .. nh - 1 pack the caller's H, then
// nb widen B's rows to a multiple of 8 elements, the rest transpose A 32 x 32 at a time (update_role reads whole
// rows of ranks). Latency bounds it: 3.5 us at 8192 x 768, rank 32, four adapters, mostly beside the plan.
struct Prepare {
    const float* H;            // [M, R] -> packed_h, scaled
    const int32_t* index;
    const float* scale;
    bf16* packed_h;
    const bf16* B;             // [b_rows, R] -> wide_b [b_rows, ld]
    bf16* wide_b;
    int64_t b_rows;
    const bf16* A;             // [count, R, K] -> turned_a [count, K, ld]
    bf16* turned_a;
    int K, ld;
    int nh, nb, na;            // CTAs of each part
};

template <int RT>
__global__ void __launch_bounds__(kThreads) prepare_kernel(const Prepare d, PlanView plan, int M, int R, int n) {
    __shared__ bf16 box[32][33];
    wait_for_previous();
    let_next_start();
    const int tid = threadIdx.x;
    int cta = blockIdx.x;
    if (cta < d.nh) {
        const int64_t pairs = (int64_t)M * (RT / 2);
        for (int64_t i = (int64_t)cta * kThreads + tid; i < pairs; i += (int64_t)d.nh * kThreads) {
            const int place = (int)(i / (RT / 2)), c = (int)(i % (RT / 2)) * 2;
            const int m = row_at(plan, place, M);
            const int a = m >= 0 && d.index ? d.index[m] : 0;
            const bool some = m >= 0 && (unsigned)a < (unsigned)n;
            const float f = some && d.scale ? d.scale[a] : 1.0f;
            uint32_t hi, lo;
            split2(some && c < R ? f * d.H[(int64_t)m * R + c] : 0.0f, some && c + 1 < R ? f * d.H[(int64_t)m * R + c + 1] : 0.0f, hi, lo);
            if (!SS1_SPAN_IN((int64_t)place * 2 * RT + RT + c, 2, (int64_t)M * 2 * RT, kSiteAdaG)) continue;
            *reinterpret_cast<uint32_t*>(d.packed_h + (int64_t)place * 2 * RT + c) = hi;
            *reinterpret_cast<uint32_t*>(d.packed_h + (int64_t)place * 2 * RT + RT + c) = lo;
        }
        return;
    }
    cta -= d.nh;
    if (cta < d.nb) {
        const int64_t size = d.b_rows * d.ld;
        for (int64_t i = (int64_t)cta * kThreads + tid; i < size; i += (int64_t)d.nb * kThreads) {
            const int64_t row = i / d.ld;
            const int r = (int)(i - row * d.ld);
            d.wide_b[i] = r < R && SS1_IN(row * R + r, d.b_rows * R, kSiteAdaB) ? d.B[row * R + r] : __float2bfloat16_rn(0.0f);
        }
        return;
    }
    cta -= d.nb;
    const int kb = (d.K + 31) / 32, rb = (d.ld + 31) / 32;      // below 2^30 boxes in all
    for (int i = cta; i < kb * rb * n; i += d.na) {
        const int k0 = i % kb * 32, r0 = i / kb % rb * 32, a = i / kb / rb;
        const bf16* from = d.A + (int64_t)a * R * d.K;
        bf16* to = d.turned_a + (int64_t)a * d.K * d.ld;
        __syncthreads();
        const int k = k0 + tid % 32;
#pragma unroll
        for (int y = 0; y < 32; y += kThreads / 32) {
            const int r = r0 + y + tid / 32;
            box[y + tid / 32][tid % 32] = r < R && k < d.K && SS1_IN(((int64_t)a * R + r) * d.K + k, (int64_t)n * R * d.K, kSiteAdaA)
                                              ? from[(int64_t)r * d.K + k] : __float2bfloat16_rn(0.0f);
        }
        __syncthreads();
        const int r = r0 + tid % 32;
#pragma unroll
        for (int y = 0; y < 32; y += kThreads / 32) {
            const int kk = k0 + y + tid / 32;
            if (kk < d.K && r < d.ld) to[(int64_t)kk * d.ld + r] = box[tid % 32][y + tid / 32];
        }
    }
}

// ---- products --------------------------------------------------------------------------------

// One cluster per tile of 128 rows, its CTAs taking equal shares of the columns: the partial
// products meet in distributed shared memory and are added in CTA order. 256 threads: warp w owns rows
// 16 w .. 16 w + 15. Stages of 64 columns: U [128][64] in 128-byte rows with the 16-byte chunks
// XOR-swizzled by the row, and T likewise: [RT][64] (TRANS false: T_a is [R, C]) or boxes of [64][64] (TRANS true: T_a
// is [C, ld]). Bound by latency, a look-up of the tile, one of its rows and nine stages a CTA: 14 us for 4096 x 4096 in
// ragged rows (34 MB, 5.1 us at the copy rate), the plan's time hidden in part by bring_ahead. H (TRANS false) is handed out in float32, so each stage's MMAs start from zero and are
// added in registers: the tensor core's own accumulation truncates, over thousands of columns by more than
// float32's rounding. G (TRANS true) only feeds bf16 results: tcgen05 multiplies out of the ring as it lies
// there and accumulates in tensor memory, one thread issuing four instructions a stage. Those sums are taken out into
// registers and begun again every 4096 columns: over all of 131,072 columns of one sign they came out 8e-4 too small.
constexpr int kStages = 4, kTakeStages = 64;

template <int RT, bool TRANS>
struct ProductsShape {
    static constexpr int u_bytes = kTile * 128;
    static constexpr int t_bytes = TRANS ? (RT + 63) / 64 * 64 * 128 : RT * 128;
    static constexpr int stage = u_bytes + t_bytes;
    static constexpr int pitch = RT + 4;                       // floats of a row of partial products
    static constexpr int ring = kStages * stage, sums = kTile * pitch * 4;
    static constexpr int smem = (ring > sums ? ring : sums) + 1024;
};

struct Products {
    const bf16* U;
    const bf16* table;
    const float* scale;      // of `packed`
    float* H;                // unscaled, by batch row; or null
    bf16* packed;
    int C, ld;
    bool table_is_new;
};

template <int RT, bool TRANS, typename W>
__device__ __forceinline__ void products_role(const Products& d, const PlanView& plan, int tile_index, uint8_t* raw, TensorState& ts, int M,
                                              int R, int n, const W& watch) {
    using S = ProductsShape<RT, TRANS>;
    const bf16 *U = d.U, *table = d.table;
    const float* scale = d.scale;
    float* H = d.H;
    bf16* packed = d.packed;
    const int C = d.C, ld = d.ld;
    // the widened B is the previous kernel's. Otherwise only the outputs' memory is shared with what ran before, and
    // every CTA still waits before it ends, so that the next kernel need not look further back than this one.
    if (d.table_is_new) wait_for_previous();
    const Tile tile = tile_of(plan, tile_index, M);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int splits = gridDim.x, split = blockIdx.x;
    if (tile.rows <= 0 || tile.adapter >= n) {                 // the whole cluster
        wait_for_previous();
        return;
    }
    if (tile.adapter < 0) {                                    // no adapter: H is 0, nobody reads the packed rows
        wait_for_previous();
        if (H)
            for (int i = split * kThreads + tid; i < tile.rows * R; i += splits * kThreads) {
                const int m = row_at(plan, tile.first + i / R, M);
                if (m >= 0 && SS1_IN((int64_t)m * R + i % R, (int64_t)M * R, kSiteAdaH)) H[(int64_t)m * R + i % R] = 0.0f;
            }
        return;
    }
    const uint32_t base = (ptx::smem_u32(raw) + 1023u) & ~1023u;
    const bf16* T = table + (int64_t)tile.adapter * C * (TRANS ? ld : R);
    const int chunks = (C + 63) / 64, per = (chunks + splits - 1) / splits;
    const int from = min(chunks, split * per), to = min(chunks, from + per);

    // this thread's pieces of a stage: a 16-byte chunk of four rows of U, and its share of T. Addresses and
    // predicates are worked out here; a stage adds one stride to each.
    const int uc = tid % 8;
    const bf16* up[4];
    bool uok[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = tid / 8 + 32 * i;
        const int m = r < tile.rows ? row_at(plan, tile.first + r, M) : -1;
        uok[i] = m >= 0;
        up[i] = U + (m >= 0 ? (int64_t)m * C : 0) + (int64_t)from * 64 + uc * 8;
    }
    constexpr int kPieces = TRANS ? 64 * (RT / 8) : RT * 8, kMine = (kPieces + kThreads - 1) / kThreads;
    const bf16* tp[kMine];
    bool tok[kMine];
    uint32_t tdst[kMine];
    int tcol[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int k = tid + i * kThreads;
        const int c = TRANS ? k / (RT / 8) : (k % 8) * 8, r = TRANS ? (k % (RT / 8)) * 8 : k / 8;
        tok[i] = k < kPieces && r < (TRANS ? ld : R);
        tcol[i] = from * 64 + c;
        tp[i] = T + (tok[i] ? (TRANS ? (int64_t)tcol[i] * ld + r : (int64_t)r * C + tcol[i]) : 0);
        tdst[i] = S::u_bytes + (TRANS ? r / 64 * 8192 + c * 128 + (((r / 8 % 8) ^ (c & 7)) << 4) : r * 128 + (((k % 8) ^ (r & 7)) << 4));
    }
    int ucol = from * 64 + uc * 8;
    auto load = [&](bool some, int slot) {      // the next stage in line
        if (some) {
            const uint32_t su = base + slot * S::stage;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = tid / 8 + 32 * i;
                const bool ok = uok[i] && ucol < C && SS1_SPAN_IN(up[i] - U, 8, (int64_t)M * C, kSiteAdaX);
                copy16(su + r * 128 + ((uc ^ (r & 7)) << 4), ok ? up[i] : U, ok);
                up[i] += 64;
            }
            ucol += 64;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const bool ok = tok[i] && tcol[i] < C && SS1_SPAN_IN(tp[i] - table, 8, (int64_t)n * C * (TRANS ? ld : R), kSiteAdaA);
                if (kPieces % kThreads == 0 || tid + i * kThreads < kPieces) copy16(su + tdst[i], ok ? tp[i] : table, ok);
                tp[i] += TRANS ? (int64_t)64 * ld : 64;
                tcol[i] += 64;
            }
        }
        ptx::cp_async_commit();
    };

#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) load(from + s < to, s);
    float* part = reinterpret_cast<float*>(raw + (base - ptx::smem_u32(raw)));   // later, over the ring's memory
    if (TRANS) {
        constexpr uint32_t kColumns = RT < 32 ? 32 : RT, kInstr = idesc_mn(RT, false, true);
        // A warp's lanes are 32 of the tile's rows; warps 4 - 7 take the upper half of the ranks, where that is 16 or more.
        constexpr int kHalf = RT < 32 ? RT : RT / 2;
        const bool reads = RT >= 32 || warp < 4;
        const int row = warp % 4 * 32 + lane, j0 = warp / 4 * kHalf;
        float sum[kHalf];
#pragma unroll
        for (int j = 0; j < kHalf; ++j) sum[j] = 0.0f;
        tensor_begin(ts, kColumns);
        const uint32_t tmem = ts.tmem;
        const bool withhold = watch.withhold == kTimeoutG && tile_index == 0 && split == 0;
        // adds what tensor memory holds, after the wait for its last product
        auto take = [&] {
            ptx::tc_fence_after();
            if (!reads) return;
#pragma unroll
            for (int j = 0; j < kHalf; j += 16) {
                uint32_t v[16];
                ptx::tmem_ld_32x32b_x16(tmem + ((uint32_t)(warp % 4 * 32) << 16) + j0 + j, v);
                ptx::tmem_ld_wait();
                ptx::tmem_ld_fence_regs<16>(v);
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[j + i] += __uint_as_float(v[i]);
            }
            ptx::tc_fence_before();
        };
        bool fresh = true;
        for (int chunk = from, slot = 0; chunk < to; ++chunk, slot = slot + 1 == kStages ? 0 : slot + 1) {
            ptx::cp_async_wait<kStages - 2>();
            ptx::fence_proxy_async_smem();
            __syncthreads();
            if (tid == 0) {
                const uint32_t su = base + slot * S::stage, stt = su + S::u_bytes;
                ptx::tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    ptx::umma_bf16_ss(tmem, desc_k(su + k * 32), desc_mn(stt + k * 2048, 8192), kInstr, !fresh || k > 0);
                if (!withhold || chunk > from) ptx::umma_commit(&ts.done[slot]);
            }
            fresh = false;
            const int last = slot == 0 ? kStages - 1 : slot - 1;      // the slot of the stage before: loaded again once read
            if (chunk > from) tensor_wait(ts, last, ((chunk - 1 - from) / kStages) & 1, watch);
            load(chunk + kStages - 1 < to, last);
            if ((chunk + 1 - from) % kTakeStages == 0 || chunk + 1 == to) {
                tensor_wait(ts, slot, ((chunk - from) / kStages) & 1, watch);
                take();
                fresh = true;      // the barrier above comes before the next product overwrites what was read
            }
        }
        ptx::cp_async_wait<0>();
        __syncthreads();
        const bool valid = tensor_fine(ts);
        if (reads) {
            float4* to_row = reinterpret_cast<float4*>(part + row * S::pitch + j0);
#pragma unroll
            for (int j = 0; j < kHalf; j += 4)
                to_row[j / 4] = valid ? make_float4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]) : make_float4(NAN, NAN, NAN, NAN);
        }
        tensor_end(ts, kColumns, watch, kTimeoutG);
    } else {
        float sum[RT / 8][4];
#pragma unroll
        for (int j = 0; j < RT / 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[j][i] = 0.0f;
        const bool busy = warp * 16 < tile.rows;
        for (int first = from; first < to; first += kStages)
#pragma unroll
            for (int s = 0; s < kStages; ++s) {
                const int chunk = first + s;
                if (chunk >= to) break;
                ptx::cp_async_wait<kStages - 2>();
                __syncthreads();
                load(chunk + kStages - 1 < to, (s + kStages - 1) % kStages);
                if (!busy) continue;
                const uint32_t su = base + s * S::stage, stt = su + S::u_bytes;
                float acc[RT / 8][4];
#pragma unroll
                for (int j = 0; j < RT / 8; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t a[4];
                    const int ar = warp * 16 + lane % 16;
                    ldsm4(a, su + ar * 128 + (((k * 2 + lane / 16) ^ (ar & 7)) << 4));
#pragma unroll
                    for (int j = 0; j < RT / 8; j += 2) {
                        uint32_t b[4];
                        const int mat = lane / 8, l8 = lane % 8, r = (j + mat / 2) * 8 + l8;
                        ldsm4(b, stt + r * 128 + (((k * 2 + mat % 2) ^ (r & 7)) << 4));
                        mma16816(acc[j], a, b[0], b[1]);
                        mma16816(acc[j + 1], a, b[2], b[3]);
                    }
                }
#pragma unroll
                for (int j = 0; j < RT / 8; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[j][i] += acc[j][i];
            }
        ptx::cp_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int j = 0; j < RT / 8; ++j) {
            const int r = warp * 16 + lane / 4, c = j * 8 + (lane % 4) * 2;
            *reinterpret_cast<float2*>(part + r * S::pitch + c) = make_float2(sum[j][0], sum[j][1]);
            *reinterpret_cast<float2*>(part + (r + 8) * S::pitch + c) = make_float2(sum[j][2], sum[j][3]);
        }
    }
    wait_for_previous();
    if (TRANS) let_next_start();           // second_gradients_kernel: what prepare_kernel wrote is complete here
    if (splits > 1) ptx::cluster_sync();
    else __syncthreads();
    const float f = scale ? scale[tile.adapter] : 1.0f;
    constexpr int kQuads = RT / 4;
    for (int i = split * kThreads + tid; i < tile.rows * kQuads; i += splits * kThreads) {
        const int r = i / kQuads, c = (i % kQuads) * 4;
        float4 u[kPortableCluster];            // all asked for before the first is added
#pragma unroll
        for (int k = 0; k < kPortableCluster; ++k)
            if (k < splits) u[k] = splits > 1 ? ld_cluster_f32x4(ptx::map_to_rank(part + r * S::pitch + c, k))
                                              : *reinterpret_cast<const float4*>(part + r * S::pitch + c);
        float v[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
        for (int k = 1; k < kPortableCluster; ++k)
            if (k < splits) { v[0] += u[k].x; v[1] += u[k].y; v[2] += u[k].z; v[3] += u[k].w; }
        const int place = tile.first + r, m = row_at(plan, place, M);
        if (H && m >= 0 && SS1_IN((int64_t)m * R, (int64_t)M * R, kSiteAdaH))
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + k < R) H[(int64_t)m * R + c + k] = v[k];
        uint2 hi, lo;
        split2(v[0] * f, v[1] * f, hi.x, lo.x);
        split2(v[2] * f, v[3] * f, hi.y, lo.y);
        if (SS1_SPAN_IN((int64_t)place * 2 * RT + RT + c, 4, (int64_t)M * 2 * RT, kSiteAdaG)) {
            *reinterpret_cast<uint2*>(packed + (int64_t)place * 2 * RT + c) = hi;
            *reinterpret_cast<uint2*>(packed + (int64_t)place * 2 * RT + RT + c) = lo;
        }
    }
    if (splits > 1) ptx::cluster_sync();   // nobody leaves while its sums are being read
}

template <int RT>
__global__ void __launch_bounds__(kThreads) products_kernel(const Products d, const Ahead ahead, PlanView plan, int M, int R, int n) {
    extern __shared__ uint8_t raw[];
    __shared__ TensorState unused;
    bring_ahead(ahead, blockIdx.y * gridDim.x + blockIdx.x, gridDim.x * gridDim.y);
    wait_for_previous();
    let_next_start();      // update_kernel reads Y and B before its own wait: they are complete here
    products_role<RT, false>(d, plan, blockIdx.y, raw, unused, M, R, n, Unwatched());
}

// ---- update ----------------------------------------------------------------------------------

// A CTA takes 128 rows of one adapter and a run of 64-column stages. A stage is in's [128][64] box in
// 128-byte rows (the two 64-byte halves of odd rows exchanged: a thread's 16-byte reads are then free of
// bank conflicts) and T's 64 rows of [C, ld], padded. Warp w owns rows 16 w .. 16 w + 15: P's parts are the A
// operand and stay in registers. Within each 32 columns T's rows are laid down so that a thread's four
// n-tiles are eight consecutive columns: it reads 16 bytes of the box, which become the MMAs' initial
// accumulators, and writes 16 bytes to `out`, four lanes 64 bytes of a row. The ring keeps three boxes
// a CTA in flight. Beside the streams the kernel has issue slots to spare only if a stage costs few
// instructions: addresses advance by one stride, ring slots are unrolled, nothing is staged twice. 4096 x 14336,
// rank 16: 42 us for 235 MB, 5.6 TB/s, 0.85 of the copy rate (five slots: 3 % slower, three CTAs of three: 4 %).
template <int RT>
struct UpdateShape {
    static constexpr int box = kTile * 128;
    static constexpr int t_pitch = RT * 2 + 16;
    static constexpr int stage = box + 64 * t_pitch;
    static constexpr int stages = 4;
    static constexpr int smem = stages * stage + 128;
};

struct Update {
    const bf16* packed;
    const bf16* table;   // [count, C, ld]
    const bf16* in;      // null: 0
    bf16* out;           // may be `in`
    int C, ld, splits;
};

template <int RT>
__device__ __forceinline__ void update_role(const Update& d, const PlanView& plan, const Tile& tile, int split, uint8_t* raw, int M,
                                            int R, int n) {
    using S = UpdateShape<RT>;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, C = d.C;
    const int chunks = (C + 63) / 64, per = (chunks + d.splits - 1) / d.splits;
    const int from = min(chunks, split * per), to = min(chunks, from + per);
    [[maybe_unused]] const int64_t total = (int64_t)M * C, tsize = (int64_t)n * C * d.ld;
    if (tile.rows <= 0 || tile.adapter >= n || from >= to || (tile.adapter < 0 && d.in == d.out)) return;
    if (tile.adapter < 0) {      // rows without an adapter are copied: a row a warp, eight vectors of a lane in flight
        constexpr int kFlight = 8;
        const int c1 = min(C, to * 64);
        for (int r = warp; r < tile.rows; r += kThreads / 32) {
            const int m = row_at(plan, tile.first + r, M);
            if (m < 0) continue;
            for (int c = from * 64 + lane * 8; c < c1; c += 32 * 8 * kFlight) {
                uint4 v[kFlight];
#pragma unroll
                for (int i = 0; i < kFlight; ++i) {
                    const int64_t at = (int64_t)m * C + c + i * 256;
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (d.in && c + i * 256 < c1 && SS1_SPAN_IN(at, 8, total, kSiteAdaY)) v[i] = *reinterpret_cast<const uint4*>(d.in + at);
                }
#pragma unroll
                for (int i = 0; i < kFlight; ++i) {
                    const int64_t at = (int64_t)m * C + c + i * 256;
                    if (c + i * 256 < c1 && SS1_SPAN_IN(at, 8, total, kSiteAdaY)) *reinterpret_cast<uint4*>(d.out + at) = v[i];
                }
            }
        }
        return;
    }
    const uint32_t base = (ptx::smem_u32(raw) + 127u) & ~127u;
    uint8_t* const ring = raw + (base - ptx::smem_u32(raw));
    const int uc = tid % 8;
    const bf16* ip[4];           // this thread's pieces of a stage: a 16-byte chunk of four rows
    bool iok[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = tid / 8 + 32 * i;
        const int m = r < tile.rows ? row_at(plan, tile.first + r, M) : -1;
        iok[i] = m >= 0 && d.in;
        ip[i] = (d.in ? d.in : d.table) + (iok[i] ? (int64_t)m * C + from * 64 + uc * 8 : 0);
    }
    constexpr int kPieces = 64 * (RT / 8), kMine = (kPieces + kThreads - 1) / kThreads;
    const bf16* tp[kMine];
    bool tok[kMine];
    uint32_t tdst[kMine];
    int tcol[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int k = tid + i * kThreads, c = k / (RT / 8), r = (k % (RT / 8)) * 8;
        tok[i] = k < kPieces && r < d.ld;
        tcol[i] = from * 64 + c;
        tp[i] = d.table + (tok[i] ? ((int64_t)tile.adapter * C + tcol[i]) * d.ld + r : 0);
        // column 8 t + 2 j + b of each 32 is row 8 j + 2 t + b
        tdst[i] = S::box + ((c & 32) | ((c & 6) << 2) | ((c & 24) >> 2) | (c & 1)) * S::t_pitch + r * 2;
    }
    int icol = from * 64 + uc * 8;
    auto load = [&](bool some, int slot) {      // the next stage in line
        if (some) {
            const uint32_t su = base + slot * S::stage;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = tid / 8 + 32 * i;
                const bool ok = iok[i] && icol < C && SS1_SPAN_IN(ip[i] - d.in, 8, total, kSiteAdaY);
                copy16(su + r * 128 + ((uc ^ ((r & 1) << 2)) << 4), ok ? ip[i] : d.table, ok);
                ip[i] += 64;
            }
            icol += 64;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const bool ok = tok[i] && tcol[i] < C && SS1_SPAN_IN(tp[i] - d.table, 8, tsize, kSiteAdaB);
                if (kPieces % kThreads == 0 || tid + i * kThreads < kPieces) copy16(su + tdst[i], ok ? tp[i] : d.table, ok);
                tp[i] += (int64_t)64 * d.ld;
                tcol[i] += 64;
            }
        }
        ptx::cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < S::stages - 1; ++s) load(from + s < to, s);
    const int g = lane / 4, t4 = lane % 4;
    bf16* op[2];                 // the two rows that this thread writes
    bool ook[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = warp * 16 + g + 8 * h;
        const int m = r < tile.rows ? row_at(plan, tile.first + r, M) : -1;
        ook[h] = m >= 0;
        op[h] = d.out + (m >= 0 ? (int64_t)m * C : 0) + from * 64 + t4 * 8;
    }
    wait_for_previous();         // `packed` is the previous kernel's; `in` and `out` are not its
    uint32_t hi[RT / 16][4], lo[RT / 16][4];
    {
        const int last = tile.first + tile.rows - 1, r0 = tile.first + warp * 16 + g;   // rows behind the end read the last one
        const uint32_t* p0 = reinterpret_cast<const uint32_t*>(d.packed + (int64_t)min(r0, last) * 2 * RT);
        const uint32_t* p1 = reinterpret_cast<const uint32_t*>(d.packed + (int64_t)min(r0 + 8, last) * 2 * RT);
#pragma unroll
        for (int k = 0; k < RT / 16; ++k) {
            hi[k][0] = p0[k * 8 + t4];
            hi[k][1] = p1[k * 8 + t4];
            hi[k][2] = p0[k * 8 + 4 + t4];
            hi[k][3] = p1[k * 8 + 4 + t4];
            lo[k][0] = p0[RT / 2 + k * 8 + t4];
            lo[k][1] = p1[RT / 2 + k * 8 + t4];
            lo[k][2] = p0[RT / 2 + k * 8 + 4 + t4];
            lo[k][3] = p1[RT / 2 + k * 8 + 4 + t4];
        }
    }
    const bool busy = warp * 16 < tile.rows;
    const uint32_t frag = (lane / 16 * 8 + lane % 8) * S::t_pitch + (lane / 8 % 2) * 16;   // this lane's row of T's fragments
    int ocol = from * 64 + t4 * 8;
    for (int first = from; first < to; first += S::stages)
#pragma unroll
        for (int s = 0; s < S::stages; ++s) {
            if (first + s >= to) break;
            ptx::cp_async_wait<S::stages - 2>();
            __syncthreads();
            load(first + s + S::stages - 1 < to, (s + S::stages - 1) % S::stages);
            if (!busy) continue;
            const uint32_t stt = base + s * S::stage + S::box + frag;
            const uint8_t* box = ring + s * S::stage + (warp * 16 + g) * 128;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float acc[4][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {     // rows g and g + 8 have the same parity
                    const uint4 y = *reinterpret_cast<const uint4*>(box + h * 8 * 128 + (((half * 4 + t4) ^ ((g & 1) << 2)) << 4));
                    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[j][2 * h] = __uint_as_float(w[j] << 16);
                        acc[j][2 * h + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                    }
                }
#pragma unroll
                for (int k = 0; k < RT / 16; ++k)
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        uint32_t b[4];
                        ldsm4(b, stt + (half * 32 + j * 8) * S::t_pitch + k * 32);
                        mma16816(acc[j], lo[k], b[0], b[1]);
                        mma16816(acc[j + 1], lo[k], b[2], b[3]);
                        mma16816(acc[j], hi[k], b[0], b[1]);
                        mma16816(acc[j + 1], hi[k], b[2], b[3]);
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(acc[j][2 * h], acc[j][2 * h + 1]);
                        w[j] = *reinterpret_cast<const uint32_t*>(&v);
                    }
                    if (ook[h] && ocol + half * 32 < C && SS1_SPAN_IN(op[h] + half * 32 - d.out, 8, total, kSiteAdaY))
                        *reinterpret_cast<uint4*>(op[h] + half * 32) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            op[0] += 64;
            op[1] += 64;
            ocol += 64;
        }
    ptx::cp_async_wait<0>();
}

template <int RT>
__global__ void __launch_bounds__(kThreads, 2) update_kernel(const Update d, PlanView plan, int M, int R, int n) {
    extern __shared__ uint8_t raw[];
    update_role<RT>(d, plan, tile_of(plan, blockIdx.y, M), blockIdx.x, raw, M, R, n);
    wait_for_previous();   // also in CTAs that left early: this grid never ends before the one before it
}

// ---- columns ---------------------------------------------------------------------------------

// A CTA takes 256 columns and a run of tiles, 32 rows a stage: U as four [32][64] boxes in swizzled
// 128-byte rows, P's packed rows as boxes of the same kind. The reduction runs over the rows, so both
// operands of D[column, rank] are read along their rows' contiguous side, as they lie: tcgen05 takes 2 x 128
// columns x (first parts, second parts) a stage from one thread, and D stays in tensor memory until the
// run comes to another adapter, when the two parts' sums are added. G and dB in one launch, 4096 x 4096 at rank 16: 18.1 us alone; dA and dX: 21.0
// (101 MB, 4.9 TB/s). (With mma.sync, whose fragments cost
// every warp transposed loads and registers, a stage took 1.2 us at rank 32: 29 us for G and dB at
// 8192 x 2304.) The tiles are dealt evenly whatever their adapters: run k's sums for adapter a go to part[k + a]
// (k and a only grow along the list, so no two share a place), or straight to `out` where the run has
// all of the adapter's tiles.
constexpr int kColCols = 256, kColRows = 32, kColSteps = kTile / kColRows;

template <int RT>
struct ColumnsShape {
    static constexpr int box = kColRows * 128;
    static constexpr int u_bytes = kColCols / 64 * box, p_boxes = (2 * RT + 63) / 64;
    static constexpr int stage = u_bytes + p_boxes * box;
    static constexpr int stages = RT <= 64 ? 4 : 3;
    static constexpr int smem = stages * stage + 1024;
    static constexpr uint32_t columns = 2 * 2 * RT;            // of tensor memory
};

struct Columns {
    const bf16* U;
    const bf16* packed;
    bf16* out;
    float* part;
    int C, cs, rs, runs;
    bool vec;           // ranks consecutive (rs 1), R a multiple of 8, `out` on a 16-byte boundary
};

// Adapter a's tiles, and the tiles of a run.
__device__ __forceinline__ int2 adapter_tiles(const PlanView& plan, int a, int M) {
    if (plan.rows == nullptr) return make_int2(0, (M + kTile - 1) / kTile);
    const int lo = min(max(plan.first_tile[a], 0), plan.max_tiles);
    return make_int2(lo, min(max(plan.first_tile[a + 1], lo), plan.max_tiles));
}
__device__ __forceinline__ int tiles_a_run(const PlanView& plan, int n, int M, int runs) {
    const int tiles = plan.rows == nullptr ? (M + kTile - 1) / kTile : min(max(plan.first_tile[n], 0), plan.max_tiles);
    return max(1, (tiles + runs - 1) / runs);
}

template <int RT, typename W>
__device__ __forceinline__ void columns_role(const Columns& d, const PlanView& plan, int range, int run, uint8_t* raw, TensorState& ts,
                                             int M, int R, int n, bool packed_is_new, const W& watch, int site) {
    using S = ColumnsShape<RT>;
    static_assert(S::stages < kSlots, "a barrier a slot, and one for the end");
    const uint32_t base = (ptx::smem_u32(raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int C = d.C, c0 = range * kColCols;
    const int tiles = adapter_tiles(plan, n - 1, M).y, per = tiles_a_run(plan, n, M, d.runs);
    const int t0 = min(tiles, run * per), t1 = min(tiles, t0 + per);
    const int steps = (t1 - t0) * kColSteps;
    static_assert(4 * kColSteps <= 32 && kColRows == 4 * (kThreads / 32), "a lane for each row of a warp's share of a tile");

    // loads: a warp brings 512 bytes of each of its four rows of a stage. Lane 4 k + i looks up row i of the
    // tile's stage k; rows are looked up a tile ahead, tiles two ahead, so that no load waits for a look-up.
    const int lc = c0 + lane * 8;
    const bool cok = lc < C;
    uint32_t udst[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = warp * 4 + i;
        udst[i] = (lane / 8) * (kColRows * 128) + r * 128 + (((lane % 8) ^ (r & 7)) << 4);
    }
    constexpr int kPieces = kColRows * (RT / 4), kMine = (kPieces + kThreads - 1) / kThreads;
    auto tile_at = [&](int t) { return t < t1 ? tile_of(plan, t, M) : Tile{-1, 0, 0}; };
    auto row_of = [&](const Tile& t) {
        const int r = (lane / 4) * kColRows + warp * 4 + lane % 4;
        return lane < 4 * kColSteps && r < t.rows ? row_at(plan, t.first + r, M) : -1;
    };
    Tile now = tile_at(t0), next = tile_at(t0 + 1), after = tile_at(t0 + 2);   // of the stage to be loaded
    int now_row = row_of(now), next_row = row_of(next);
    auto load_u = [&](int step, int slot) {
        if (step < steps) {
            const uint32_t su = base + slot * S::stage;
            const int k = step % kColSteps;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = __shfl_sync(0xFFFFFFFFu, now_row, k * 4 + i);
                const int64_t at = (int64_t)m * C + lc;
                const bool ok = m >= 0 && cok && SS1_SPAN_IN(at, 8, (int64_t)M * C, kSiteAdaX);
                copy16(su + udst[i], ok ? d.U + at : d.U, ok);
            }
        }
    };
    auto load_p = [&](const Tile& tile, int step, int slot) {
        if (step < steps) {
            const uint32_t sp = base + slot * S::stage + S::u_bytes;
            const int k = step % kColSteps;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int e = tid + i * kThreads, r = e / (RT / 4), c = (e % (RT / 4)) * 8;
                const int64_t at = (int64_t)(tile.first + k * kColRows + r) * 2 * RT + c;
                const bool ok = k * kColRows + r < tile.rows && SS1_SPAN_IN(at, 8, (int64_t)M * 2 * RT, kSiteAdaG);
                if (kPieces % kThreads == 0 || e < kPieces)
                    copy16(sp + c / 64 * S::box + r * 128 + (((c / 8 % 8) ^ (r & 7)) << 4), ok ? d.packed + at : d.packed, ok);
            }
        }
        ptx::cp_async_commit();
    };
    auto advance = [&](int step) {
        if (step < steps && step % kColSteps == kColSteps - 1) {
            now = next;
            now_row = next_row;
            next = after;
            next_row = row_of(next);
            after = tile_at(t0 + step / kColSteps + 3);
        }
    };

    int adapter = now.adapter, next_adapter = adapter;
    static_assert(S::stages - 1 <= kColSteps, "the first stages lie in the first tile");
    const Tile head = now;
    for (int s = 0; s < S::stages - 1; ++s) load_u(s, s);
    if (packed_is_new) wait_for_previous();      // P is the previous kernel's, U and the plan are not
    for (int s = 0; s < S::stages - 1; ++s) load_p(head, s, s);
    for (int s = 0; s < S::stages - 1; ++s) advance(s);
    tensor_begin(ts, S::columns);
    const uint32_t tmem = ts.tmem;
    const bool withhold = watch.withhold == site && range == 0 && run == 0;
    constexpr uint32_t kInstr = idesc_mn(2 * RT, true, true);
    const int64_t size = (int64_t)C * R;
    bool fresh = true;
    for (int step = 0, slot = 0;; ++step) {
        if (step % kColSteps == 0 || step == steps) {       // a tile begins, or the run ends
            const int a = step < steps ? next_adapter : -1;
            if (step + kColSteps < steps) next_adapter = tile_of(plan, t0 + step / kColSteps + 1, M).adapter;
            if (a != adapter && (unsigned)adapter < (unsigned)n) {
                tensor_wait(ts, slot == 0 ? S::stages - 1 : slot - 1, ((step - 1) / S::stages) & 1, watch);
                ptx::tc_fence_after();
                const bool valid = tensor_fine(ts);
                const int2 own = adapter_tiles(plan, adapter, M);
                const bool whole = own.x >= t0 && own.y <= t1;
                const int64_t place = whole ? adapter * size : (int64_t)(run + adapter) * size;
                [[maybe_unused]] const int64_t all = (whole ? n : d.runs + n) * size;
                const int c = c0 + warp * 32 + lane;        // warps 0 - 3: the first 128 columns, lane by lane; 4 - 7 the others
                const uint32_t from_lane = tmem + warp / 4 * 2 * RT + ((uint32_t)(warp % 4 * 32) << 16);
                for (int j = 0; j < RT && j < R; j += 16) {
                    uint32_t hi[16], lo[16];
                    ptx::tmem_ld_32x32b_x16(from_lane + j, hi);
                    ptx::tmem_ld_32x32b_x16(from_lane + RT + j, lo);
                    ptx::tmem_ld_wait();
                    ptx::tmem_ld_fence_regs<16>(hi);
                    ptx::tmem_ld_fence_regs<16>(lo);
                    float v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = valid ? __uint_as_float(hi[i]) + __uint_as_float(lo[i]) : NAN;
                    if (c >= C) continue;
                    const int64_t first = place + (int64_t)c * d.cs + (int64_t)j * d.rs;
                    if (d.vec) {       // a lane's ranks lie together: element by element each would be a sector of its own
#pragma unroll
                        for (int i = 0; i < 16; i += 8) {
                            if (j + i >= R || !SS1_SPAN_IN(first + i, 8, all, kSiteAdaPart)) continue;
                            if (whole) {
                                Raw8<bf16> r;
                                const float w[8] = {v[i], v[i + 1], v[i + 2], v[i + 3], v[i + 4], v[i + 5], v[i + 6], v[i + 7]};
                                r.set(w);
                                r.store(d.out + first + i);
                            } else {
                                *reinterpret_cast<float4*>(d.part + first + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                                *reinterpret_cast<float4*>(d.part + first + i + 4) = make_float4(v[i + 4], v[i + 5], v[i + 6], v[i + 7]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int64_t at = first + (int64_t)i * d.rs;
                            if (j + i >= R || !SS1_IN(at, all, kSiteAdaPart)) continue;
                            if (whole) d.out[at] = __float2bfloat16_rn(v[i]);
                            else d.part[at] = v[i];
                        }
                    }
                }
                ptx::tc_fence_before();
                fresh = true;      // the barrier below comes before the next product overwrites what was read
            }
            adapter = a;
            if (step == steps) break;
        }
        ptx::cp_async_wait<S::stages - 2>();
        ptx::fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            const uint32_t su = base + slot * S::stage, sp = su + S::u_bytes;
            ptx::tc_fence_after();
#pragma unroll
            for (int k = 0; k < kColRows / 16; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    ptx::umma_bf16_ss(tmem + h * 2 * RT, desc_mn(su + h * 2 * S::box + k * 2048, S::box), desc_mn(sp + k * 2048, S::box), kInstr,
                                      !fresh || k > 0);
            if (!withhold || step > 0) ptx::umma_commit(&ts.done[slot]);
        }
        fresh = false;
        const int last = slot == 0 ? S::stages - 1 : slot - 1;        // the slot of the step before: loaded again once read
        if (step > 0) tensor_wait(ts, last, ((step - 1) / S::stages) & 1, watch);
        load_u(step + S::stages - 1, last);
        load_p(now, step + S::stages - 1, last);
        advance(step + S::stages - 1);
        slot = slot == S::stages - 1 ? 0 : slot + 1;
    }
    ptx::cp_async_wait<0>();
    tensor_end(ts, S::columns, watch, site);
}

// G and dB in one launch: both read dY (from HBM once: the other reader finds it in L2). The first `tiles` rows of
// the grid are G's clusters; the CTAs behind them, as many as dB has, take its columns and runs.
template <int RT>
constexpr int first_smem() {
    return ColumnsShape<RT>::smem > ProductsShape<RT, true>::smem ? ColumnsShape<RT>::smem : ProductsShape<RT, true>::smem;
}

template <int RT, typename W>
__global__ void __launch_bounds__(kThreads, RT <= 64 ? 2 : 1) first_gradients_kernel(const Products g, int tiles, const Columns db, int nb,
                                                                                     PlanView plan, int M, int R, int n,
                                                                                     const W watch) {
    extern __shared__ uint8_t raw[];
    __shared__ TensorState ts;
    if ((int)blockIdx.y < tiles) {
        products_role<RT, true>(g, plan, blockIdx.y, raw, ts, M, R, n, watch);
    } else {
        wait_for_previous();      // the packed H
        let_next_start();
        const int k = ((int)blockIdx.y - tiles) * gridDim.x + blockIdx.x, ranges = (db.C + kColCols - 1) / kColCols;
        if (k < nb) columns_role<RT>(db, plan, k % ranges, k / ranges, raw, ts, M, R, n, false, watch, kTimeoutDb);
    }
}

// dA and dX in one launch: both need G, but their first loads, of X, dX and A, do not wait for it (300 x 1024 x 1024 16.2 -> 15.3
// us, 8192 x 768 x 2304 47.1 -> 46.5, 4096 x 4096 x 14336 63.8 -> 65.4). CTAs 0 .. na - 1 take dA, the rest dX.
template <int RT>
constexpr int second_smem() {
    return ColumnsShape<RT>::smem > UpdateShape<RT>::smem ? ColumnsShape<RT>::smem : UpdateShape<RT>::smem;
}

template <int RT, typename W>
__global__ void __launch_bounds__(kThreads, RT <= 64 ? 2 : 1) second_gradients_kernel(const Columns da, int na, const Update dx,
                                                                                      PlanView plan, int M, int R, int n,
                                                                                      const W watch) {
    // CTAs of both launches may share an SM: their tensor memory has room, or shared memory for one of them only. (The decode
    // kernel, which holds tensor memory while it waits, takes 166 KB of shared memory or more: never beside one of these.)
    static_assert(RT <= 64 ? 2 * ColumnsShape<RT>::columns <= 512 && first_smem<RT>() + 2 * second_smem<RT>() > 232448
                           : first_smem<RT>() + second_smem<RT>() > 232448, "512 columns an SM");
    extern __shared__ uint8_t raw[];
    __shared__ TensorState ts;
    let_next_start();      // its successors wait first thing
    const int i = blockIdx.x;
    if (i < na) {
        const int ranges = (da.C + kColCols - 1) / kColCols;
        columns_role<RT>(da, plan, i % ranges, i / ranges, raw, ts, M, R, n, true, watch, kTimeoutDa);
    } else {
        update_role<RT>(dx, plan, tile_of(plan, (i - na) / dx.splits, M), (i - na) % dx.splits, raw, M, R, n);
    }
    wait_for_previous();   // also in CTAs that left early
}

// Latency again: 6 us alone for 4 + 4 MB of partial sums, of which its launch and look-ups are hidden.
// The runs' partial sums, in run order, for the adapters whose tiles lie in several runs; zeros for those
// without rows. y = 0: dA, 1: dB; z: adapters in turn.
struct Sums {
    const float* part[2];
    bf16* out[2];
    int64_t size[2];         // elements of one adapter
    int runs[2];
};
__global__ void __launch_bounds__(kThreads) add_kernel(const Sums s, PlanView plan, int M, int n) {
    __shared__ int16_t runs_of[kMaxCount][2];
    wait_for_previous();
    const int w = blockIdx.y;
    if (s.out[w] == nullptr) return;
    const int64_t size = s.size[w];
    const int per = tiles_a_run(plan, n, M, s.runs[w]);
    // every adapter's first and last run, all looked up at once
    for (int a = threadIdx.x; a < n; a += kThreads) {
        const int2 own = adapter_tiles(plan, a, M);
        const int lo = own.x / per, hi = own.y > own.x ? min((own.y - 1) / per, s.runs[w] - 1) : lo - 1;
        runs_of[a][0] = (int16_t)lo;
        runs_of[a][1] = (int16_t)hi;
    }
    __syncthreads();
    const bool vec = size % 4 == 0;
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4; i < size; i += (int64_t)gridDim.x * kThreads * 4)
        for (int a = blockIdx.z; a < n; a += gridDim.z) {
            const int lo = runs_of[a][0], hi = runs_of[a][1];
            if (lo == hi) continue;          // written by the run itself
            const float* p = s.part[w] + (int64_t)(lo + a) * size + i;
            bf16* to = s.out[w] + a * size + i;
            if (vec) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                for (int k = lo; k <= hi; ++k, p += size) {
                    const float4 u = *reinterpret_cast<const float4*>(p);
                    v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
                }
                to[0] = __float2bfloat16_rn(v.x);
                to[1] = __float2bfloat16_rn(v.y);
                to[2] = __float2bfloat16_rn(v.z);
                to[3] = __float2bfloat16_rn(v.w);
            } else {
                for (int e = 0; e < 4 && i + e < size; ++e) {
                    float v = 0.0f;
                    for (int k = lo; k <= hi; ++k) v += p[(int64_t)(k - lo) * size + e];
                    to[e] = __float2bfloat16_rn(v);
                }
            }
        }
}

// ---- launches --------------------------------------------------------------------------------

int tiles_at_most(const Call& c) { return c.plan.rows ? c.plan.max_tiles : (int)((c.M + kTile - 1) / kTile); }

// Shares of the columns for `tiles` row tiles: about `ctas` CTAs in all, at least four 64-column stages each.
int stage_splits(int64_t C, int tiles, int ctas, int most) {
    const int stages = (int)((C + 255) / 256);
    int s = ctas / tiles;
    s = s > stages ? stages : s;
    s = s > most ? most : s;
    return s < 1 ? 1 : s;
}

// CTAs of each part of the backward's two launches
constexpr int kFirstCtas = 148, kColumnsCtas = 148, kUpdateCtas = 296;
constexpr int kRunTiles = 32;      // of a run in dA or dB, about

// H packed and A transposed where the pointers are given, B widened where R is no multiple of 8; *B and *ld: B as
// the kernels read it.
template <int RT>
cudaError_t prepare(const Call& c, const MmaSpace& w, const float* H, bool turn_a, bool with_b, const void** B, int* ld,
                    bool* launched, cudaStream_t st) {
    Prepare d = {};
    d.ld = (c.R + 7) / 8 * 8;
    *ld = d.ld;
    *B = c.B;
    auto ctas = [](int64_t work) { return (int)(work > 592 ? 592 : work); };
    if (H) {
        d.H = H; d.index = c.index; d.scale = c.scale; d.packed_h = (bf16*)w.packed_h;
        d.nh = ctas((c.M * (RT / 2) + kThreads - 1) / kThreads);
    }
    if (with_b && c.R % 8) {
        d.B = (const bf16*)c.B; d.wide_b = (bf16*)w.wide_b; d.b_rows = (int64_t)c.n * c.N;
        d.nb = ctas((d.b_rows * d.ld + kThreads - 1) / kThreads);
        *B = w.wide_b;
    }
    if (turn_a) {
        d.A = (const bf16*)c.A; d.turned_a = (bf16*)w.turned_a; d.K = (int)c.K;
        d.na = ctas((c.K + 31) / 32 * ((d.ld + 31) / 32) * c.n);
    }
    *launched = d.nh + d.nb + d.na > 0;
    if (!*launched) return cudaSuccess;
    return launch_dependent(&prepare_kernel<RT>, dim3((unsigned)(d.nh + d.nb + d.na)), dim3(kThreads), 0, st, d, c.plan, (int)c.M, c.R, c.n);
}

// A launch of clusters of (x, 1, 1) CTAs; `dependent`: it may start while the previous kernel drains.
template <typename... P, typename... A>
cudaError_t launch_clusters(void (*fn)(P...), dim3 grid, int x, size_t smem, bool dependent, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)x;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = dependent ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
}

template <int RT>
cudaError_t forward_rt(const Call& c, const void* X, const void* Y, void* out, float* H, const MmaSpace& w, cudaStream_t st) {
    using SP = ProductsShape<RT, false>;
    using SU = UpdateShape<RT>;
    auto* pfn = &products_kernel<RT>;
    auto* ufn = &update_kernel<RT>;
    int ld;
    const void* B;
    bool launched;
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(pfn), SP::smem);
    if (e == cudaSuccess) e = smem_attr_once(reinterpret_cast<const void*>(ufn), SU::smem);
    if (e == cudaSuccess) e = prepare<RT>(c, w, nullptr, false, true, &B, &ld, &launched, st);
    if (e != cudaSuccess) return e;
    const int tiles = tiles_at_most(c);
    const int psplits = stage_splits(c.K, tiles, 296, kPortableCluster), usplits = stage_splits(c.N, tiles, 296, 1 << 20);
    const Products p{(const bf16*)X, (const bf16*)c.A, c.scale, H, (bf16*)w.packed_g, (int)c.K, c.R, false};
    e = launch_clusters(pfn, dim3((unsigned)psplits, (unsigned)tiles), psplits, SP::smem, true, st, p, ahead_of(c, X, Y), c.plan, (int)c.M, c.R, c.n);
    if (e != cudaSuccess) return e;
    const Update d{(const bf16*)w.packed_g, (const bf16*)B, (const bf16*)Y, (bf16*)out, (int)c.N, ld, usplits};
    return launch_dependent(ufn, dim3((unsigned)usplits, (unsigned)tiles), dim3(kThreads), SU::smem, st, d, c.plan, (int)c.M, c.R, c.n);
}

template <int RT, typename W>
cudaError_t backward_rt(const Call& c, const void* dY, const void* X, const float* H, const void* dX_in, void* dX, void* dA, void* dB,
                        const MmaSpace& w, const W& watch, cudaStream_t st) {
    auto* fn1 = &first_gradients_kernel<RT, W>;
    auto* fn2 = &second_gradients_kernel<RT, W>;
    int ld;
    const void* B;
    bool prepared;
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(fn1), first_smem<RT>());
    if (e == cudaSuccess) e = smem_attr_once(reinterpret_cast<const void*>(fn2), second_smem<RT>());
    if (e == cudaSuccess) e = prepare<RT>(c, w, dB ? H : nullptr, dX != nullptr, dX || dA, &B, &ld, &prepared, st);
    if (e != cudaSuccess) return e;
    const int rb = mma_runs(c.M, c.N, c.n), ra = mma_runs(c.M, c.K, c.n);
    const Columns db{(const bf16*)dY, (const bf16*)w.packed_h, (bf16*)dB, w.part_b, (int)c.N, c.R, 1, rb, c.R % 8 == 0 && aligned(dB, 16)};
    const Columns da{(const bf16*)X, (const bf16*)w.packed_g, (bf16*)dA, w.part_a, (int)c.K, 1, (int)c.K, ra, false};
    const int nb = dB ? (db.C + kColCols - 1) / kColCols * rb : 0;
    const int na = dA ? (da.C + kColCols - 1) / kColCols * ra : 0;
    const int tiles = tiles_at_most(c), gtiles = dX || dA ? tiles : 0;
    const int splits = stage_splits(c.N, tiles, kFirstCtas, kPortableCluster);
    const Products g{(const bf16*)dY, (const bf16*)B, c.scale, nullptr, (bf16*)w.packed_g, (int)c.N, ld, B != c.B};
    e = launch_clusters(fn1, dim3((unsigned)splits, (unsigned)(gtiles + (nb + splits - 1) / splits)), splits, first_smem<RT>(), prepared, st,
                        g, gtiles, db, nb, c.plan, (int)c.M, c.R, c.n, watch);
    if (e != cudaSuccess) return e;
    if (dX || dA) {
        const Update dx{(const bf16*)w.packed_g, (const bf16*)w.turned_a, (const bf16*)dX_in, (bf16*)dX, (int)c.K, ld,
                        stage_splits(c.K, tiles, kUpdateCtas, 1 << 20)};
        const int64_t ctas = (int64_t)na + (dX ? (int64_t)tiles * dx.splits : 0);
        e = launch_dependent(fn2, dim3((unsigned)ctas), dim3(kThreads), second_smem<RT>(), st, da, na, dx, c.plan, (int)c.M, c.R, c.n, watch);
        if (e != cudaSuccess) return e;
    }
    if (!dA && !dB) return cudaSuccess;
    Sums s = {};
    if (dA) { s.part[0] = da.part; s.out[0] = da.out; s.size[0] = (int64_t)c.K * c.R; s.runs[0] = ra; }
    if (dB) { s.part[1] = db.part; s.out[1] = db.out; s.size[1] = (int64_t)c.N * c.R; s.runs[1] = rb; }
    const int64_t size = s.size[0] > s.size[1] ? s.size[0] : s.size[1], blocks = (size + 4 * kThreads - 1) / (4 * kThreads);
    return launch_dependent(&add_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096), 2, (unsigned)(c.n < 4 ? c.n : 4)),
                            dim3(kThreads), 0, st, s, c.plan, (int)c.M, c.n);
}

}  // namespace

int mma_rank(int R) { return R <= 16 ? 16 : (R <= 32 ? 32 : (R <= 64 ? 64 : 128)); }

int mma_runs(int64_t M, int64_t C, int n) {
    // one CTA an SM for each gradient, since both launches do other work beside (two: 8192 x 768 x 2304, rank 32, 57 us
    // instead of 48), and a run for every tile while they are few (two tiles a run: 2048 x 768 x 2304 37 us instead of 29)
    const int64_t ranges = (C + kColCols - 1) / kColCols, tiles = M / kTile;
    int64_t s = kColumnsCtas / ranges;
    const int64_t most = tiles + n;
    s = s > most ? most : s;
    // Tensor memory truncates its sums: 9 runs of 524,288 rows of one sign came out 3e-4 too small, as much as
    // bf16 rounds by. So a run has about 32 tiles at most (4096 rows: 1e-5), within what the grid can count.
    int64_t least = (tiles + (n < tiles ? n : tiles) + kRunTiles - 1) / kRunTiles;
    if (least > 32000 / ranges) least = 32000 / ranges;
    s = s < least ? least : s;
    return (int)(s < 1 ? 1 : s);
}

cudaError_t mma_forward(const Call& c, const void* X, const void* Y, void* out, float* H, const MmaSpace& w, cudaStream_t st) {
    switch (mma_rank(c.R)) {
        case 16: return forward_rt<16>(c, X, Y, out, H, w, st);
        case 32: return forward_rt<32>(c, X, Y, out, H, w, st);
        case 64: return forward_rt<64>(c, X, Y, out, H, w, st);
        default: return forward_rt<128>(c, X, Y, out, H, w, st);
    }
}

namespace {
template <typename W>
cudaError_t backward_of(const Call& c, const void* dY, const void* X, const float* H, const void* dX_in, void* dX, void* dA, void* dB,
                        const MmaSpace& w, const W& watch, cudaStream_t st) {
    switch (mma_rank(c.R)) {
        case 16: return backward_rt<16>(c, dY, X, H, dX_in, dX, dA, dB, w, watch, st);
        case 32: return backward_rt<32>(c, dY, X, H, dX_in, dX, dA, dB, w, watch, st);
        case 64: return backward_rt<64>(c, dY, X, H, dX_in, dX, dA, dB, w, watch, st);
        default: return backward_rt<128>(c, dY, X, H, dX_in, dX, dA, dB, w, watch, st);
    }
}
}  // namespace

cudaError_t mma_backward(const Call& c, const void* dY, const void* X, const float* H, const void* dX_in, void* dX, void* dA, void* dB,
                         const MmaSpace& w, const Watch* test, cudaStream_t st) {
    return test ? backward_of(c, dY, X, H, dX_in, dX, dA, dB, w, *test, st) : backward_of(c, dY, X, H, dX_in, dX, dA, dB, w, Unwatched(), st);
}

cudaError_t mma_status(int32_t* detail) {
    int32_t v = 0;
    const int32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof v);
    if (e == cudaSuccess && v != 0) e = cudaMemcpyToSymbol(g_status, &zero, sizeof zero);
    if (e == cudaSuccess) *detail = v;
    return e;
}

}  // namespace ada
}  // namespace ss1
