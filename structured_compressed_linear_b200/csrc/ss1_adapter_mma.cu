// The adapters' products on the tensor cores (bf16): three kernels make up both passes.
//
//   products : P[m, r] = sum_c U[m, c] T_a[c, r]             H = X A^T (forward), G = s dY B (backward)
//   update   : out[m, c] = in[m, c] + sum_r P[m, r] T_a[c, r]    out = Y + s H B^T,   dX + G A
//   columns  : D_a[c, r] = sum_m U[m, c] P[m, r]             dA = G^T X,        dB = dY^T (s H)
//
// Each streams its [rows, columns] matrix once and does 2 R (4 R where P is split) flops for each
// element: at ranks up to 32 that is below what mma.sync sustains beside a full HBM stream, so these
// kernels are built as streams (cp.async rings, 16-byte vectors, rows gathered through the plan by
// their own pointers) with register-accumulator MMAs inside, and not around tcgen05 tiles, whose
// 128-wide accumulators an adapter's few columns would leave idle.
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

constexpr int kThreads = 256;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
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

struct Tile {
    int adapter, first, rows;   // adapter -1: rows without one
};
__device__ __forceinline__ Tile tile_of(const PlanView& plan, int i, int M) {
    if (plan.rows == nullptr) return Tile{0, i * kTile, min(kTile, M - i * kTile)};
    const int4 t = plan.tiles[i];
    return Tile{t.x, t.y, min(t.z, M - t.y)};   // a plan of another batch cannot lead past M places
}
// The batch row at a place of the plan, -1 if there is none.
__device__ __forceinline__ int row_at(const PlanView& plan, int place, int M) {
    const int m = plan.rows == nullptr ? place : plan.rows[place];
    return (unsigned)m < (unsigned)M ? m : -1;
}

// ---- products --------------------------------------------------------------------------------

// One cluster per tile of 128 rows, its CTAs taking equal shares of the columns: the partial
// products meet in distributed shared memory and are added in CTA order. 256 threads: warp w owns rows
// 16 w .. 16 w + 15. Stages of 64 columns: U [128][64] in 128-byte rows with the 16-byte chunks
// XOR-swizzled by the row, and T either [RT][64] likewise (TRANS false: T_a is [R, C]) or [64][RT] in padded
// rows (TRANS true: T_a is [C, ld]). Each stage's MMAs start from zero and are added in float32:
// the tensor core's own accumulation truncates, over thousands of columns by more than float32's rounding.
constexpr int kStages = 4;

template <int RT, bool TRANS>
struct ProductsShape {
    static constexpr int u_bytes = kTile * 128;
    static constexpr int t_pitch = TRANS ? RT * 2 + 16 : 128;
    static constexpr int t_bytes = TRANS ? 64 * t_pitch : RT * 128;
    static constexpr int stage = u_bytes + t_bytes;
    static constexpr int pitch = RT + 4;                       // floats of a row of partial products
    static constexpr int ring = kStages * stage, sums = kTile * pitch * 4;
    static constexpr int smem = (ring > sums ? ring : sums) + 128;
};

template <int RT, bool TRANS>
__global__ void __launch_bounds__(kThreads) products_kernel(const bf16* __restrict__ U, const bf16* __restrict__ table, int ld,
                                                            const float* __restrict__ scale, PlanView plan, float* __restrict__ H,
                                                            bf16* __restrict__ packed, bool scale_packed, int M, int C, int R,
                                                            int n) {
    using S = ProductsShape<RT, TRANS>;
    extern __shared__ uint8_t raw[];
    let_next_start();
    const Tile tile = tile_of(plan, blockIdx.y, M);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int splits = gridDim.x, split = blockIdx.x;
    if (tile.rows <= 0 || tile.adapter >= n) return;           // the whole cluster
    if (tile.adapter < 0) {                                    // no adapter: H is 0, nobody reads the packed rows
        if (H)
            for (int i = split * kThreads + tid; i < tile.rows * R; i += splits * kThreads) {
                const int m = row_at(plan, tile.first + i / R, M);
                if (m >= 0 && SS1_IN((int64_t)m * R + i % R, (int64_t)M * R, kSiteAdaH)) H[(int64_t)m * R + i % R] = 0.0f;
            }
        return;
    }
    const uint32_t base = (ptx::smem_u32(raw) + 127u) & ~127u;
    const bf16* T = table + (int64_t)tile.adapter * C * (TRANS ? ld : R);
    const int chunks = (C + 63) / 64, per = (chunks + splits - 1) / splits;
    const int from = min(chunks, split * per), to = min(chunks, from + per);

    // this thread's four rows of a stage: one 16-byte chunk of each
    const bf16* urow[4];
    const int uc = tid % 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = tid / 8 + 32 * i;
        const int m = r < tile.rows ? row_at(plan, tile.first + r, M) : -1;
        urow[i] = m >= 0 ? U + (int64_t)m * C : nullptr;
    }
    auto load = [&](int chunk, int slot) {
        if (chunk < to) {
            const uint32_t su = base + slot * S::stage, stt = su + S::u_bytes;
            const int c0 = chunk * 64;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = tid / 8 + 32 * i, c = c0 + uc * 8;
                const bool ok = urow[i] && c < C && SS1_SPAN_IN(urow[i] + c - U, 8, (int64_t)M * C, kSiteAdaX);
                copy16(su + r * 128 + ((uc ^ (r & 7)) << 4), ok ? urow[i] + c : U, ok);
            }
            if (TRANS) {
                constexpr int cw = RT / 8;
                for (int i = tid; i < 64 * cw; i += kThreads) {
                    const int c = c0 + i / cw, r = (i % cw) * 8;
                    const bool ok = c < C && r < ld && SS1_SPAN_IN(T + (int64_t)c * ld + r - table, 8, (int64_t)n * C * ld, kSiteAdaB);
                    copy16(stt + (i / cw) * S::t_pitch + r * 2, ok ? T + (int64_t)c * ld + r : table, ok);
                }
            } else {
                for (int i = tid; i < RT * 8; i += kThreads) {
                    const int r = i / 8, c = c0 + (i % 8) * 8;
                    const bool ok = r < R && c < C && SS1_SPAN_IN(T + (int64_t)r * C + c - table, 8, (int64_t)n * C * R, kSiteAdaA);
                    copy16(stt + r * 128 + (((i % 8) ^ (r & 7)) << 4), ok ? T + (int64_t)r * C + c : table, ok);
                }
            }
        }
        ptx::cp_async_commit();
    };

    float sum[RT / 8][4];
#pragma unroll
    for (int j = 0; j < RT / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[j][i] = 0.0f;
    for (int s = 0; s < kStages - 1; ++s) load(from + s, s);
    const bool busy = warp * 16 < tile.rows;
    for (int chunk = from; chunk < to; ++chunk) {
        ptx::cp_async_wait<kStages - 2>();
        __syncthreads();
        load(chunk + kStages - 1, (chunk - from + kStages - 1) % kStages);
        if (!busy) continue;
        const uint32_t su = base + ((chunk - from) % kStages) * S::stage, stt = su + S::u_bytes;
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
                const int mat = lane / 8, l8 = lane % 8;
                if (TRANS) {
                    ldsm4_trans(b, stt + (k * 16 + (mat % 2) * 8 + l8) * S::t_pitch + (j + mat / 2) * 16);
                } else {
                    const int r = (j + mat / 2) * 8 + l8;
                    ldsm4(b, stt + r * 128 + (((k * 2 + mat % 2) ^ (r & 7)) << 4));
                }
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
    // the partial products over the ring's memory
    float* part = reinterpret_cast<float*>(raw + (base - ptx::smem_u32(raw)));
#pragma unroll
    for (int j = 0; j < RT / 8; ++j) {
        const int r = warp * 16 + lane / 4, c = j * 8 + (lane % 4) * 2;
        *reinterpret_cast<float2*>(part + r * S::pitch + c) = make_float2(sum[j][0], sum[j][1]);
        *reinterpret_cast<float2*>(part + (r + 8) * S::pitch + c) = make_float2(sum[j][2], sum[j][3]);
    }
    if (splits > 1) ptx::cluster_sync();
    else __syncthreads();
    const float f = scale ? scale[tile.adapter] : 1.0f;
    const int pairs = tile.rows * (RT / 2);
    for (int i = split * kThreads + tid; i < pairs; i += splits * kThreads) {
        const int r = i / (RT / 2), c = (i % (RT / 2)) * 2;
        float x = 0.0f, y = 0.0f;
        if (splits > 1) {
            for (int k = 0; k < splits; ++k) {
                const uint32_t at = ptx::map_to_rank(part + r * S::pitch + c, k);
                x += ptx::ld_cluster_f32(at);
                y += ptx::ld_cluster_f32(at + 4);
            }
        } else {
            x = part[r * S::pitch + c];
            y = part[r * S::pitch + c + 1];
        }
        const int place = tile.first + r, m = row_at(plan, place, M);
        if (H && m >= 0 && SS1_IN((int64_t)m * R, (int64_t)M * R, kSiteAdaH)) {
            if (c < R) H[(int64_t)m * R + c] = x;
            if (c + 1 < R) H[(int64_t)m * R + c + 1] = y;
        }
        if (scale_packed) { x *= f; y *= f; }
        uint32_t hi, lo;
        split2(x, y, hi, lo);
        if (SS1_SPAN_IN((int64_t)place * 2 * RT + RT + c, 2, (int64_t)M * 2 * RT, kSiteAdaG)) {
            *reinterpret_cast<uint32_t*>(packed + (int64_t)place * 2 * RT + c) = hi;
            *reinterpret_cast<uint32_t*>(packed + (int64_t)place * 2 * RT + RT + c) = lo;
        }
    }
    if (splits > 1) ptx::cluster_sync();   // nobody leaves while its sums are being read
}

// packed[i] = scale[a] H[rows[i]] in two parts, for an H that the caller brings.
template <int RT>
__global__ void __launch_bounds__(kThreads) pack_kernel(const float* __restrict__ H, const int32_t* __restrict__ index,
                                                        const float* __restrict__ scale, PlanView plan, bf16* __restrict__ packed,
                                                        int M, int R, int n) {
    let_next_start();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int place = (int)(i / (RT / 2)), c = (int)(i % (RT / 2)) * 2;
    if (place >= M) return;
    const int m = row_at(plan, place, M);
    const int a = m >= 0 && index ? index[m] : 0;
    const bool some = m >= 0 && (unsigned)a < (unsigned)n;
    const float f = some && scale ? scale[a] : 1.0f;
    uint32_t hi, lo;
    split2(some && c < R ? f * H[(int64_t)m * R + c] : 0.0f, some && c + 1 < R ? f * H[(int64_t)m * R + c + 1] : 0.0f, hi, lo);
    *reinterpret_cast<uint32_t*>(packed + (int64_t)place * 2 * RT + c) = hi;
    *reinterpret_cast<uint32_t*>(packed + (int64_t)place * 2 * RT + RT + c) = lo;
}

// out[i, 0 .. ld) = in[i, 0 .. R) with zeros behind it: rows of a rank that is no multiple of 8.
__global__ void __launch_bounds__(kThreads) widen_kernel(const bf16* __restrict__ in, bf16* __restrict__ out, int64_t rows, int R,
                                                         int ld) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= rows * ld) return;
    const int64_t row = i / ld;
    const int r = (int)(i % ld);
    out[i] = r < R ? in[row * R + r] : __float2bfloat16_rn(0.0f);
}

// ---- update ----------------------------------------------------------------------------------

// A CTA takes 128 rows of one adapter x kCols columns. T's columns lie in shared memory as [column][RT]
// in padded rows, ordered so that a thread's four n-tiles give it eight consecutive columns: it
// reads and writes `in` and `out` in 16-byte vectors straight from its accumulators, 64 bytes of a
// row by each four lanes. P's parts are the MMAs' A operand and stay in registers.
template <int RT>
constexpr int update_cols() { return RT <= 32 ? 512 : 256; }
template <int RT>
constexpr int update_smem() { return update_cols<RT>() * (RT * 2 + 16); }

template <int RT>
__global__ void __launch_bounds__(kThreads, RT <= 32 ? 3 : 2) update_kernel(const bf16* __restrict__ packed,
                                                                            const bf16* __restrict__ table, int64_t tstride,
                                                                            int cs, int rs, PlanView plan, const bf16* in, bf16* out,
                                                                            int M, int C, int R, int n) {
    constexpr int kCols = update_cols<RT>(), kPitch = RT * 2 + 16;
    extern __shared__ __align__(16) uint8_t raw[];
    const Tile tile = tile_of(plan, blockIdx.y, M);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int c0 = blockIdx.x * kCols;
    // every CTA waits before it leaves, so that this grid never ends before the one before it
    if (tile.rows <= 0 || tile.adapter >= n || (tile.adapter < 0 && in == out)) {
        wait_for_previous();
        return;
    }
    if (tile.adapter < 0) {      // rows without an adapter are copied
        wait_for_previous();
        for (int i = tid; i < tile.rows * (kCols / 8); i += kThreads) {
            const int m = row_at(plan, tile.first + i / (kCols / 8), M), c = c0 + (i % (kCols / 8)) * 8;
            if (m < 0 || c >= C || !SS1_SPAN_IN((int64_t)m * C + c, 8, (int64_t)M * C, kSiteAdaY)) continue;
            const int64_t at = (int64_t)m * C + c;
            *reinterpret_cast<uint4*>(out + at) = in ? *reinterpret_cast<const uint4*>(in + at) : make_uint4(0, 0, 0, 0);
        }
        return;
    }
    // shared-memory row of column n: within each 32, column 8 t + 2 j + b is row 8 j + 2 t + b
    const bf16* T = table + (int64_t)tile.adapter * tstride;
    const int cols = min(kCols, C - c0);
    auto slot = [](int c) { return (c & ~31) | ((c & 6) << 2) | ((c & 24) >> 2) | (c & 1); };
    if (rs == 1 && R % 8 == 0 && cs % 8 == 0) {      // T_a rows of R: 16-byte pieces
        for (int i = tid; i < kCols * (RT / 8); i += kThreads) {
            const int c = i / (RT / 8), r = (i % (RT / 8)) * 8;
            const bool ok = c < cols && r < R && SS1_SPAN_IN(T + (int64_t)(c0 + c) * cs + r - table, 8, n * tstride, kSiteAdaB);
            *reinterpret_cast<uint4*>(raw + slot(c) * kPitch + r * 2) =
                ok ? *reinterpret_cast<const uint4*>(T + (int64_t)(c0 + c) * cs + r) : make_uint4(0, 0, 0, 0);
        }
    } else {                                         // transposed, or odd ranks: consecutive threads along the contiguous side
        for (int i = tid; i < kCols * RT; i += kThreads) {
            const int c = rs == 1 ? i / RT : i % kCols, r = rs == 1 ? i % RT : i / kCols;
            const bool ok = c < cols && r < R && SS1_IN(T + (int64_t)(c0 + c) * cs + (int64_t)r * rs - table, n * tstride, kSiteAdaA);
            *reinterpret_cast<bf16*>(raw + slot(c) * kPitch + r * 2) =
                ok ? T[(int64_t)(c0 + c) * cs + (int64_t)r * rs] : __float2bfloat16_rn(0.0f);
        }
    }
    const int g = lane / 4, t4 = lane % 4;
    const int r0 = warp * 16 + g;
    const int m0 = r0 < tile.rows ? row_at(plan, tile.first + r0, M) : -1;
    const int m1 = r0 + 8 < tile.rows ? row_at(plan, tile.first + r0 + 8, M) : -1;
    __syncthreads();
    wait_for_previous();
    if (warp * 16 >= tile.rows) return;
    uint32_t hi[RT / 16][4], lo[RT / 16][4];
    {
        const int last = tile.first + tile.rows - 1;   // rows behind the tile's end read its last one; they are not written
        const uint32_t* p0 = reinterpret_cast<const uint32_t*>(packed + (int64_t)min(tile.first + r0, last) * 2 * RT);
        const uint32_t* p1 = reinterpret_cast<const uint32_t*>(packed + (int64_t)min(tile.first + r0 + 8, last) * 2 * RT);
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
    const uint32_t base = ptx::smem_u32(raw);
    constexpr int kBatch = 4;      // 32-column steps whose vectors are in flight together
    for (int q0 = 0; q0 * 32 < cols; q0 += kBatch) {
        uint4 y[kBatch][2];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int c = c0 + (q0 + q) * 32 + t4 * 8;
            y[q][0] = y[q][1] = make_uint4(0, 0, 0, 0);
            if (in && c < C) {
                if (m0 >= 0 && SS1_SPAN_IN((int64_t)m0 * C + c, 8, (int64_t)M * C, kSiteAdaY))
                    y[q][0] = *reinterpret_cast<const uint4*>(in + (int64_t)m0 * C + c);
                if (m1 >= 0 && SS1_SPAN_IN((int64_t)m1 * C + c, 8, (int64_t)M * C, kSiteAdaY))
                    y[q][1] = *reinterpret_cast<const uint4*>(in + (int64_t)m1 * C + c);
            }
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            if ((q0 + q) * 32 >= cols) break;
            float acc[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
#pragma unroll
            for (int k = 0; k < RT / 16; ++k)
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    uint32_t b[4];
                    ldsm4(b, base + ((q0 + q) * 32 + (j + lane / 16) * 8 + lane % 8) * kPitch + (k * 2 + (lane / 8) % 2) * 16);
                    mma16816(acc[j], lo[k], b[0], b[1]);
                    mma16816(acc[j], hi[k], b[0], b[1]);
                    mma16816(acc[j + 1], lo[k], b[2], b[3]);
                    mma16816(acc[j + 1], hi[k], b[2], b[3]);
                }
            const int c = c0 + (q0 + q) * 32 + t4 * 8;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int m = h ? m1 : m0;
                if (m < 0 || c >= C) continue;
                Raw8<bf16> v;
                v.a = y[q][h];
                float f[8];
                v.get(f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[2 * j] += acc[j][2 * h];
                    f[2 * j + 1] += acc[j][2 * h + 1];
                }
                v.set(f);
                if (SS1_SPAN_IN((int64_t)m * C + c, 8, (int64_t)M * C, kSiteAdaY)) v.store(out + (int64_t)m * C + c);
            }
        }
    }
}

// ---- columns ---------------------------------------------------------------------------------

// A CTA takes 256 columns of one adapter and a share of its rows, 64 rows a stage: U as four
// [64][64] boxes in swizzled 128-byte rows, P's packed rows in padded ones. Warp w owns columns
// 32 w .. 32 w + 31: U transposed out of shared memory is the A operand (column x row), P the B
// operand, and the sums over all rows stay in registers.
constexpr int kColCols = 256, kColRows = 64;

template <int RT>
struct ColumnsShape {
    static constexpr int u_bytes = kColRows * kColCols * 2;
    static constexpr int p_pitch = RT * 4 + 16;
    static constexpr int stage = u_bytes + kColRows * p_pitch;
    static constexpr int stages = RT <= 64 ? 4 : 3;
    static constexpr int smem = stages * stage + 128;
};

struct Columns {
    const bf16* U;
    const bf16* packed;
    bf16* out;
    float* part;        // partial sums of the shares, or null: one share, which writes `out`
    int C, cs, rs, shares;
};

template <int RT>
__global__ void __launch_bounds__(kThreads) columns_kernel(const Columns d, PlanView plan, int M, int R, int n) {
    using S = ColumnsShape<RT>;
    extern __shared__ uint8_t raw[];
    wait_for_previous();
    const uint32_t base = (ptx::smem_u32(raw) + 127u) & ~127u;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int a = blockIdx.y, share = blockIdx.z, C = d.C;
    const int c0 = blockIdx.x * kColCols;
    const int begin = plan.rows ? max(0, plan.first[a]) : 0, end = plan.rows ? min(M, plan.first[a + 1]) : M;
    const int steps = end > begin ? (end - begin + kColRows - 1) / kColRows : 0, per = (steps + d.shares - 1) / d.shares;
    const int from = min(steps, share * per), to = min(steps, from + per);

    auto load = [&](int step, int slot) {
        if (step < to) {
            const uint32_t su = base + slot * S::stage, sp = su + S::u_bytes;
            const int r0 = begin + step * kColRows;
#pragma unroll
            for (int i = 0; i < kColRows * kColCols / 8 / kThreads; ++i) {
                const int r = warp + i * 8, c = c0 + lane * 8;       // a warp brings 512 bytes of one row
                const int m = r0 + r < end ? row_at(plan, r0 + r, M) : -1;
                const bool ok = m >= 0 && c < C && SS1_SPAN_IN((int64_t)m * C + c, 8, (int64_t)M * C, kSiteAdaX);
                copy16(su + (lane / 8) * (kColRows * 128) + r * 128 + (((lane % 8) ^ (r & 7)) << 4), ok ? d.U + (int64_t)m * C + c : d.U,
                       ok);
            }
            for (int i = tid; i < kColRows * (RT / 4); i += kThreads) {
                const int r = i / (RT / 4), c = (i % (RT / 4)) * 8;
                const bool ok = r0 + r < end && SS1_SPAN_IN((int64_t)(r0 + r) * 2 * RT + c, 8, (int64_t)M * 2 * RT, kSiteAdaG);
                copy16(sp + r * S::p_pitch + c * 2, ok ? d.packed + (int64_t)(r0 + r) * 2 * RT + c : d.packed, ok);
            }
        }
        ptx::cp_async_commit();
    };

    float acc[2][RT / 8][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < RT / 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[h][j][i] = 0.0f;
    for (int s = 0; s < S::stages - 1; ++s) load(from + s, s);
    const bool busy = c0 + warp * 32 < C;
    for (int step = from; step < to; ++step) {
        ptx::cp_async_wait<S::stages - 2>();
        __syncthreads();
        load(step + S::stages - 1, (step - from + S::stages - 1) % S::stages);
        if (!busy) continue;
        const uint32_t su = base + ((step - from) % S::stages) * S::stage, sp = su + S::u_bytes;
        const int mat = lane / 8, l8 = lane % 8;
#pragma unroll
        for (int k = 0; k < kColRows / 16; ++k) {
            uint32_t u[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = k * 16 + (mat / 2) * 8 + l8, chunk = warp * 4 + h * 2 + mat % 2;
                ldsm4_trans(u[h], su + (chunk / 8) * (kColRows * 128) + r * 128 + (((chunk % 8) ^ (r & 7)) << 4));
            }
#pragma unroll
            for (int j = 0; j < RT / 8; j += 2) {
                uint32_t b[4], l[4];
                const uint32_t at = sp + (k * 16 + (mat % 2) * 8 + l8) * S::p_pitch + (j + mat / 2) * 16;
                ldsm4_trans(b, at);
                ldsm4_trans(l, at + RT * 2);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mma16816(acc[h][j], u[h], l[0], l[1]);
                    mma16816(acc[h][j], u[h], b[0], b[1]);
                    mma16816(acc[h][j + 1], u[h], l[2], l[3]);
                    mma16816(acc[h][j + 1], u[h], b[2], b[3]);
                }
            }
        }
    }
    ptx::cp_async_wait<0>();
    if (!busy) return;
    const int64_t size = (int64_t)n * C * R;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < RT / 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + warp * 32 + h * 16 + lane / 4 + (i / 2) * 8, r = j * 8 + (lane % 4) * 2 + i % 2;
                if (c >= C || r >= R) continue;
                const int64_t at = (int64_t)a * C * R + (int64_t)c * d.cs + (int64_t)r * d.rs;
                if (!SS1_IN(at, size, kSiteAdaPart)) continue;
                if (d.part) d.part[share * size + at] = acc[h][j][i];
                else d.out[at] = __float2bfloat16_rn(acc[h][j][i]);
            }
}

// out[i] = the shares' partial sums, in share order, for both gradients (y = 0, 1).
struct Sums {
    const float* part[2];
    bf16* out[2];
    int64_t size[2];
    int shares[2];
};
__global__ void __launch_bounds__(kThreads) add_kernel(const Sums s) {
    wait_for_previous();
    const int w = blockIdx.y;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (s.part[w] == nullptr || i >= s.size[w]) return;
    float v = 0.0f;
    for (int k = 0; k < s.shares[w]; ++k) v += s.part[w][k * s.size[w] + i];
    s.out[w][i] = __float2bfloat16_rn(v);
}

// ---- launches --------------------------------------------------------------------------------

int tiles_at_most(const Call& c) { return c.plan.rows ? c.plan.max_tiles : (int)((c.M + kTile - 1) / kTile); }

template <int RT, bool TRANS>
cudaError_t products(const Call& c, const void* U, const void* table, int ld, int64_t C, float* H, void* packed,
                     bool scale_packed, cudaStream_t st) {
    using S = ProductsShape<RT, TRANS>;
    auto* fn = &products_kernel<RT, TRANS>;
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(fn), S::smem);
    if (e != cudaSuccess) return e;
    const int tiles = tiles_at_most(c);
    // two CTAs for each of 148 SMs, at least four stages of columns each, clusters of a portable size
    int splits = 296 / tiles;
    const int most = (int)((C + 255) / 256);
    splits = splits > most ? most : splits;
    splits = splits < 1 ? 1 : (splits > 8 ? 8 : splits);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)splits, (unsigned)tiles);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)splits;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, (const bf16*)U, (const bf16*)table, ld, c.scale, c.plan, H, (bf16*)packed, scale_packed,
                              (int)c.M, (int)C, c.R, c.n);
}

template <int RT>
cudaError_t update(const Call& c, const void* packed, const void* table, int64_t C, int cs, int rs, const void* in, void* out,
                   cudaStream_t st) {
    auto* fn = &update_kernel<RT>;
    const cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(fn), update_smem<RT>());
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((C + update_cols<RT>() - 1) / update_cols<RT>()), (unsigned)tiles_at_most(c));
    return launch_dependent(fn, grid, dim3(kThreads), update_smem<RT>(), st, (const bf16*)packed, (const bf16*)table,
                            (int64_t)C * c.R, cs, rs, c.plan, (const bf16*)in, (bf16*)out, (int)c.M, (int)C, c.R, c.n);
}

template <int RT>
cudaError_t columns(const Call& c, const Columns& d, cudaStream_t st) {
    using S = ColumnsShape<RT>;
    auto* fn = &columns_kernel<RT>;
    const cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(fn), S::smem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((d.C + kColCols - 1) / kColCols), (unsigned)c.n, (unsigned)d.shares);
    return launch_dependent(fn, grid, dim3(kThreads), S::smem, st, d, c.plan, (int)c.M, c.R, c.n);
}

template <int RT>
cudaError_t forward_rt(const Call& c, const void* X, const void* Y, void* out, float* H, void* packed, cudaStream_t st) {
    const cudaError_t e = products<RT, false>(c, X, c.A, c.R, c.K, H, packed, true, st);
    if (e != cudaSuccess) return e;
    return update<RT>(c, packed, c.B, c.N, c.R, 1, Y, out, st);
}

template <int RT>
cudaError_t backward_rt(const Call& c, const void* dY, const void* X, const float* H, const void* dX_in, void* dX, void* dA, void* dB,
                        const MmaSpace& w, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (dB) {
        const int64_t pairs = c.M * (RT / 2);
        pack_kernel<RT><<<(unsigned)((pairs + kThreads - 1) / kThreads), kThreads, 0, st>>>(H, c.index, c.scale, c.plan, (bf16*)w.packed_h,
                                                                                          (int)c.M, c.R, c.n);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess && (dX || dA)) {
        const void* B = c.B;
        int ld = c.R;
        if (c.R % 8) {
            ld = (c.R + 7) / 8 * 8;
            const int64_t size = (int64_t)c.n * c.N * ld;
            widen_kernel<<<(unsigned)((size + kThreads - 1) / kThreads), kThreads, 0, st>>>((const bf16*)c.B, (bf16*)w.wide_b,
                                                                                           (int64_t)c.n * c.N, c.R, ld);
            e = cudaGetLastError();
            B = w.wide_b;
        }
        if (e == cudaSuccess) e = products<RT, true>(c, dY, B, ld, c.N, nullptr, w.packed_g, true, st);
    }
    Sums s = {};
    if (e == cudaSuccess && dB) {
        const int shares = mma_shares(c.M, c.N, c.n);
        const Columns d{(const bf16*)dY, (const bf16*)w.packed_h, (bf16*)dB, shares > 1 ? w.part_b : nullptr, (int)c.N, c.R, 1, shares};
        e = columns<RT>(c, d, st);
        s.part[1] = d.part; s.out[1] = d.out; s.size[1] = (int64_t)c.n * c.N * c.R; s.shares[1] = shares;
    }
    if (e == cudaSuccess && dX) e = update<RT>(c, w.packed_g, c.A, c.K, 1, (int)c.K, dX_in, dX, st);
    if (e == cudaSuccess && dA) {
        const int shares = mma_shares(c.M, c.K, c.n);
        const Columns d{(const bf16*)X, (const bf16*)w.packed_g, (bf16*)dA, shares > 1 ? w.part_a : nullptr, (int)c.K, 1, (int)c.K, shares};
        e = columns<RT>(c, d, st);
        s.part[0] = d.part; s.out[0] = d.out; s.size[0] = (int64_t)c.n * c.K * c.R; s.shares[0] = shares;
    }
    if (e == cudaSuccess && (s.part[0] || s.part[1])) {
        const int64_t size = s.size[0] > s.size[1] ? s.size[0] : s.size[1];
        e = launch_dependent(&add_kernel, dim3((unsigned)((size + kThreads - 1) / kThreads), 2), dim3(kThreads), 0, st, s);
    }
    return e;
}

}  // namespace

int mma_rank(int R) { return R <= 16 ? 16 : (R <= 32 ? 32 : (R <= 64 ? 64 : 128)); }

int mma_shares(int64_t M, int64_t C, int n) {
    // one CTA for each of 148 SMs, at least four stages of rows a share
    const int64_t ctas = (C + kColCols - 1) / kColCols * n;
    int64_t s = 148 / ctas;
    const int64_t most = M / (4 * kColRows);
    s = s > most ? most : s;
    return (int)(s < 1 ? 1 : (s > 32 ? 32 : s));
}

cudaError_t mma_forward(const Call& c, const void* X, const void* Y, void* out, float* H, void* packed, cudaStream_t st) {
    switch (mma_rank(c.R)) {
        case 16: return forward_rt<16>(c, X, Y, out, H, packed, st);
        case 32: return forward_rt<32>(c, X, Y, out, H, packed, st);
        case 64: return forward_rt<64>(c, X, Y, out, H, packed, st);
        default: return forward_rt<128>(c, X, Y, out, H, packed, st);
    }
}

cudaError_t mma_backward(const Call& c, const void* dY, const void* X, const float* H, const void* dX_in, void* dX, void* dA, void* dB,
                         const MmaSpace& w, cudaStream_t st) {
    switch (mma_rank(c.R)) {
        case 16: return backward_rt<16>(c, dY, X, H, dX_in, dX, dA, dB, w, st);
        case 32: return backward_rt<32>(c, dY, X, H, dX_in, dX, dA, dB, w, st);
        case 64: return backward_rt<64>(c, dY, X, H, dX_in, dX, dA, dB, w, st);
        default: return backward_rt<128>(c, dY, X, H, dX_in, dX, dA, dB, w, st);
    }
}

}  // namespace ada
}  // namespace ss1
