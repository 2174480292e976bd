// Internal declarations of the low-rank adapters' kernels (ss1_adapter.cu).
#pragma once

#include "ss1_ops.cuh"

namespace ss1 {
namespace ada {

constexpr int kTile = 128;                               // rows of a tile
constexpr int kMaxRank = SS1_ADAPTER_MAX_RANK;
constexpr int kMaxCount = SS1_ADAPTER_MAX_COUNT;

// The rows of a batch by adapter, in device memory: adapter a's rows are rows[first[a] .. first[a + 1]),
// the rows without one come last (group `count`). tiles: {adapter or -1, first place in rows, rows, 0};
// adapter a's are tiles[first_tile[a] .. first_tile[a + 1]), those behind the last one have no rows. All
// null where every row uses adapter 0.
struct PlanView {
    int32_t* first;         // [count + 2]
    int32_t* first_tile;    // [count + 2]
    int4* tiles;
    int32_t* rows;
    int max_tiles;
};

inline int max_tiles(int64_t M, int n) { return (int)(M / kTile) + n + 1; }   // each group's last tile may be short
size_t plan_bytes(int64_t M, int n);
PlanView plan_view(void* plan, int64_t M, int n);
cudaError_t launch_plan(const int32_t* index, int64_t M, int n, PlanView plan, cudaStream_t st);

struct Call {
    const void *A, *B;
    const float* scale;
    const int32_t* index;
    PlanView plan;
    int64_t M, K, N;
    int R, n;
    bool planned;            // the plan's kernel is part of this call
};

// Shares of an adapter's rows in the sums of dA and dB (general path).
int general_shares(int64_t M, int64_t C, int R, int n);

// Forward for a few rows (ss1_adapter_rows.cu): K, N and R multiples of 8, 16-byte aligned rows, either type.
cudaError_t rows_forward(const Call& c, const void* X, const void* Y, void* out, float* H, int dtype, cudaStream_t st);

// Tensor-core path (ss1_adapter_mma.cu): bf16, K and N multiples of 8, 16-byte aligned rows.
struct MmaSpace {
    void *packed_g, *packed_h;   // [M][2][mma_rank(R)] bf16 in plan order, two parts each: s H (forward) or G; s H beside it
    void* wide_b;                // B with rows of a multiple of 8 elements, where R is none
    void* turned_a;              // A transposed, [count][K][R rounded up to 8]
    float *part_a, *part_b;      // the runs' partial dA and dB
};
int mma_rank(int R);                             // R as the kernels pad it
int mma_runs(int64_t M, int64_t C, int n);       // runs of tiles in dA or dB with C columns
cudaError_t mma_forward(const Call& c, const void* X, const void* Y, void* out, float* H, const MmaSpace& w, cudaStream_t st);
// The test of a wait that runs out: waits end after limit_ns, and the first CTA at `withhold` (a TimeoutSite) does not announce
// the products of its first stage.
struct Watch {
    uint64_t limit_ns;
    int withhold;
};
enum TimeoutSite : int { kTimeoutG = 1, kTimeoutDb, kTimeoutDa };     // with the kernel id 4 in the status word
constexpr int32_t kStatusKernelAdapter = 4;
cudaError_t mma_backward(const Call& c, const void* dY, const void* X, const float* H, const void* dX_in, void* dX, void* dA, void* dB,
                         const MmaSpace& w, const Watch* test, cudaStream_t st);
cudaError_t mma_status(int32_t* detail);         // reads and clears the current device's status word

}  // namespace ada
}  // namespace ss1
