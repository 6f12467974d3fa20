// Lookup of rows by token or species and its gradient, gfx950.
//
//   y[i] = a T[index[i]],   dT[v] = a sum of dy[i] over the rows i with index[i] = v
//
// Both are bound by memory.  The lookup is a copy whose rows are found by an index.
//
// The gradient is a sum over runs of equal entries in the sorted order of the rows
// (perm).  The sorted positions are cut evenly, whatever the runs are: every L lanes
// take `len` positions in turn and add their rows in registers; a run that lies
// within them is written at once.  A run that goes on is joined with its neighbours'
// parts in LDS, and one that leaves the workgroup's positions leaves fp32 sums
// for a second kernel, which adds them in order.  So a token that holds a tenth
// of all rows costs no more than rare ones, and no sum depends on timing.
// Further workgroups of the same launch write the zeros of entries without a row.
//
// Measured on MI355X (a copy reaches 5.15 TB/s):
//  - lookup of 65536 rows of 1024 in bf16: 33.6 us, 5.0 TB/s of 168 MB (38 in a kernel that
//    takes rows of any alignment too).
//  - gradient of 16 entries over 647170 rows of 32 in fp32: 20.8 and 4.8 us, 4.0 TB/s of
//    85 MB: two rounds of dependent reads (positions, rows) in five workgroups a unit.
//    With the entries read through the index 25 us: its lines come in anew for
//    every entry.  Parts of runs added one behind the other in LDS: 29 and 8.1 us.
//  - gradient of 32000 entries over 16384 rows of 2048 in bf16: 32 and 4.8 us, 6.2 TB/s
//    of 198 MB, most of it zeros.
//  - gradient of 21 entries over 42993 rows of 461 in bf16: 16 and 9 us (464: 15 and 9);
//    29 and 40 with sums of the row's own width, column by column.
#include "zs_launch.h"
#include "zs_layers_internal.h"
#include "zs_row.h"

namespace zs {

namespace {

// ---- lookup -------------------------------------------------------------------

template <typename T>
struct EmbedParams {
    const T* table;
    const int64_t* index;
    int64_t ldt, n_rows, n_entries;
    int c;
    float scale;
    bool vec;
    T* y;
};

// L lanes copy a row chunk by chunk, U rows at a time.
// WHOLE: rows on 16 bytes of whole chunks.
template <typename T, int L, int U, bool WHOLE>
__global__ __launch_bounds__(256) void zs_embed_kernel(const EmbedParams<T> p) {
    constexpr int V = Chunk<T>::V, kRows = 256 / L;
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    const int chunks = (p.c + V - 1) / V;
    for (int64_t base = int64_t(blockIdx.x) * kRows * U; base < p.n_rows;
         base += int64_t(gridDim.x) * kRows * U) {
        int64_t from[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = base + u * kRows + slot;
            const int64_t at = row < p.n_rows ? p.index[row] : -1;
            from[u] = at >= 0 && at < p.n_entries ? at : -1;
        }
        for (int chunk = l; chunk < chunks; chunk += L) {
            u32x4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                v[u] = from[u] < 0 ? u32x4{0, 0, 0, 0}
                                   : load_raw(p.table + from[u] * p.ldt, chunk, p.c, WHOLE);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = base + u * kRows + slot;
                if (row >= p.n_rows) continue;
                float f[V];
                Chunk<T>::unpack(settled<T>(v[u], chunk, p.c, WHOLE), f);
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] *= p.scale;
                // a row of no entry is +0 whatever the scale's sign
                store_any(p.y + row * p.c, chunk, p.c, WHOLE,
                          from[u] < 0 ? v[u] : Chunk<T>::pack(f));
            }
        }
    }
}

template <typename T, int L, bool WHOLE>
hipError_t run_embed(const EmbedParams<T>& p, hipStream_t stream) {
    constexpr int kRows = 256 / L;
    const int64_t one = (p.n_rows + kRows - 1) / kRows;
    // four rows at a time where that still leaves several workgroups for every unit
    if (one >= 4096) {
        const int64_t want = (one + 3) / 4;
        zs_embed_kernel<T, L, 4, WHOLE>
            <<<unsigned(want < 1 << 20 ? want : 1 << 20), 256, 0, stream>>>(p);
    } else {
        zs_embed_kernel<T, L, 1, WHOLE><<<unsigned(one), 256, 0, stream>>>(p);
    }
    return hipGetLastError();
}

template <typename T, int L>
hipError_t run_embed(const EmbedParams<T>& p, hipStream_t stream) {
    return p.vec ? run_embed<T, L, true>(p, stream) : run_embed<T, L, false>(p, stream);
}

bool on16(const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; }

template <typename T>
hipError_t embed(const EmbedArgs& a, hipStream_t stream) {
    constexpr int V = Chunk<T>::V;
    EmbedParams<T> p{};
    p.table = static_cast<const T*>(a.table), p.index = a.index, p.ldt = a.ldt;
    p.n_rows = a.n_rows, p.n_entries = a.n_entries, p.c = a.c, p.scale = a.scale;
    p.y = static_cast<T*>(a.y);
    p.vec = a.c % V == 0 && a.ldt % V == 0 && on16(a.table) && on16(a.y);
    const int chunks = (a.c + V - 1) / V;
    if (chunks <= 1) return run_embed<T, 1>(p, stream);
    if (chunks <= 2) return run_embed<T, 2>(p, stream);
    if (chunks <= 4) return run_embed<T, 4>(p, stream);
    if (chunks <= 8) return run_embed<T, 8>(p, stream);
    if (chunks <= 16) return run_embed<T, 16>(p, stream);
    if (chunks <= 32) return run_embed<T, 32>(p, stream);
    if (chunks <= 64) return run_embed<T, 64>(p, stream);
    if (chunks <= 128) return run_embed<T, 128>(p, stream);
    return run_embed<T, 256>(p, stream);
}

// ---- gradient -----------------------------------------------------------------

constexpr int kThreads = 256;
constexpr int kMaxPositions = 2048;   // of a workgroup (their rows and entries lie in LDS)
constexpr int kMaxLen = 64;           // positions in turn
constexpr int kAhead = 8;             // rows whose loads are in flight together
constexpr int kFewEntries = 1024;     // entries whose offsets fit in LDS

template <typename T>
struct GradParams {
    const T* gy;
    const int64_t* index;
    const int32_t *offsets, *perm;
    int64_t ldg, n_rows, n_entries;
    int c, len, blocks;      // positions in turn; column blocks of 64 chunks
    int64_t pieces;          // workgroups along the positions
    int64_t block0;          // number of the launch's first workgroup
    int zero_rows;           // entries that a workgroup looks at for zeros
    float scale;
    bool vec;
    T* grad;
    float* sums;      // [pieces][2][whole chunks]: of the run that enters a piece, of the one that leaves it
    int32_t* leaves;  // [pieces]: the entry whose run starts in the piece and leaves it, or -1
};

// First and last sorted position that belongs to an entry, inside [0, n_rows].
template <typename T>
__device__ inline void positions(const GradParams<T>& p, int64_t& first, int64_t& last) {
    first = p.offsets[0], last = p.offsets[p.n_entries];
    first = first < 0 ? 0 : first;
    last = last > p.n_rows ? p.n_rows : last;
}

template <typename T>
__device__ inline void store_row(const GradParams<T>& p, int64_t entry, int chunk,
                                 const float (&v)[Chunk<T>::V]) {
    constexpr int V = Chunk<T>::V;
    float f[V];
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = v[i] * p.scale;
    store_any(p.grad + entry * p.c, chunk, p.c, p.vec, Chunk<T>::pack(f));
}
// fp32 sums of a chunk's columns, in rows of whole chunks.
template <int V>
__device__ inline void store_sums(float* row, int chunk, int chunks, const float (&v)[V]) {
    if (chunk >= chunks) return;
#pragma unroll
    for (int i = 0; i < V; i += 4)
        *reinterpret_cast<f32x4*>(row + chunk * V + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
}
template <int V>
__device__ inline void load_sums(const float* row, int chunk, int chunks, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const f32x4 t = chunk < chunks ? *reinterpret_cast<const f32x4*>(row + chunk * V + i)
                                       : f32x4{0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < 4; ++q) v[i + q] = t[q];
    }
}

// The entry whose positions hold q: the last v with offsets[v] <= q (of equal offsets
// the one that has rows), offsets in LDS.
__device__ inline int entry_at(const int32_t* offsets, int n_entries, int64_t q) {
    int lo = 0, hi = n_entries - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (offsets[mid] <= q) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <typename T, int L, bool FEW>
__global__ __launch_bounds__(kThreads) void zs_embed_grad_kernel(const GradParams<T> p) {
    constexpr int V = Chunk<T>::V, W = kThreads / L;
    constexpr int kPositions = W * kMaxLen < kMaxPositions ? W * kMaxLen : kMaxPositions;
    __shared__ int32_t rows[kPositions];
    __shared__ int32_t entry_of[kPositions + 2];   // one position before and behind
    __shared__ int32_t offsets[FEW ? kFewEntries : 1];
    __shared__ __align__(16) float head[W][L * V];
    __shared__ bool through[W];
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    const int chunks = (p.c + V - 1) / V, width = chunks * V;
    const int64_t work = p.pieces * p.blocks, block = p.block0 + blockIdx.x;
    if (block >= work) {   // zeros
        const int64_t v0 = (block - work) * p.zero_rows;
        for (int r = slot; r < p.zero_rows; r += W) {
            const int64_t v = v0 + r;
            if (v >= p.n_entries || p.offsets[v] < p.offsets[v + 1]) continue;
            for (int chunk = l; chunk < chunks; chunk += L)
                store_any(p.grad + v * p.c, chunk, p.c, p.vec, u32x4{0, 0, 0, 0});
        }
        return;
    }
    const int64_t piece = block / p.blocks;
    const int chunk = int(block % p.blocks) * L + l;
    const int count = W * p.len;
    int64_t first, last;
    positions(p, first, last);
    const int64_t q0 = first + piece * count;
    if constexpr (FEW) {
        for (int v = threadIdx.x; v < p.n_entries; v += kThreads) offsets[v] = p.offsets[v];
        __syncthreads();
    }
    for (int i = int(threadIdx.x) - 1; i <= count; i += kThreads) {
        const int64_t q = q0 + i;
        int64_t row = -1, v = -1;
        if (q >= first && q < last) {
            row = p.perm ? p.perm[q] : q;
            if (row < 0 || row >= p.n_rows) row = -1;
            if constexpr (FEW) v = entry_at(offsets, int(p.n_entries), q);
            else if (row >= 0) v = p.index[row];
            if (row < 0 || v < 0 || v >= p.n_entries) v = -1;
        }
        entry_of[i + 1] = int32_t(v);
        if (i >= 0 && i < count) rows[i] = int32_t(row);
    }
    __syncthreads();
    const int i0 = slot * p.len, i1 = i0 + p.len;
    float acc[V], entering[V];   // of the run in hand; of one that entered and ended here
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = entering[j] = 0.0f;
    int32_t cur = entry_of[i0 + 1];
    const bool entered = cur >= 0 && cur == entry_of[i0];
    bool inside = entered;   // the run in hand is the one that entered
    for (int i = i0; i < i1; i += kAhead) {
        u32x4 raw[kAhead];
        int32_t at[kAhead];
        const auto load = [&](bool vec) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                at[j] = entry_of[i + j + 1];
                raw[j] = at[j] < 0 ? u32x4{0, 0, 0, 0}
                                   : load_raw<T, true>(p.gy + int64_t(rows[i + j]) * p.ldg, chunk,
                                                       p.c, vec);
            }
        };
        if (p.vec) load(true);
        else load(false);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (at[j] != cur) {   // a run ends here
                if (inside) {
#pragma unroll
                    for (int e = 0; e < V; ++e) entering[e] = acc[e];
                } else if (cur >= 0) {
                    store_row(p, cur, chunk, acc);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] = 0.0f;
                cur = at[j];
                inside = false;
            }
            float f[V];
            Chunk<T>::unpack(settled<T>(raw[j], chunk, p.c, p.vec), f);
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += f[e];
        }
    }
    const bool goes_on = cur >= 0 && cur == entry_of[i1 + 1];
    const bool starts = goes_on && !inside;   // a run starts among these positions and goes on
    if (inside) {
#pragma unroll
        for (int e = 0; e < V; ++e) entering[e] = acc[e];
    } else if (cur >= 0 && !goes_on) {
        store_row(p, cur, chunk, acc);
    }
    // The parts of runs that enter lanes' positions, each added up to where its run ends
    // or leaves the workgroup, in log2(W) steps: after the step of distance d a part holds
    // what lies 2 d slots on, as far as its run goes.
    bool open = inside && goes_on;
#pragma unroll
    for (int d = 1; d < W; d *= 2) {
#pragma unroll
        for (int e = 0; e < V; ++e) head[slot][l * V + e] = entering[e];
        if (l == 0) through[slot] = open;
        __syncthreads();
        if (open && slot + d < W) {
#pragma unroll
            for (int e = 0; e < V; ++e) entering[e] += head[slot + d][l * V + e];
            open = through[slot + d];
        }
        __syncthreads();
    }
#pragma unroll
    for (int e = 0; e < V; ++e) head[slot][l * V + e] = entering[e];
    if (l == 0) through[slot] = open;
    __syncthreads();
    if (slot == 0 && entered) store_sums<V>(p.sums + piece * 2 * width, chunk, chunks, entering);
    bool leaves = false;
    if (starts) {
        leaves = true;
        if (slot + 1 < W) {
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += head[slot + 1][l * V + e];
            leaves = through[slot + 1];
        }
        if (leaves) store_sums<V>(p.sums + (piece * 2 + 1) * width, chunk, chunks, acc);
        else store_row(p, cur, chunk, acc);
    }
    // one run at most starts here and leaves
    const bool any = __syncthreads_or(leaves);
    if (p.pieces > 1 && l == 0 && (leaves || (slot == 0 && !any)))
        p.leaves[piece] = leaves ? cur : -1;
}

// Adds the sums of a run that goes over several pieces, in order: L lanes a row and
// W parts, joined in LDS.
template <typename T, int L>
__global__ __launch_bounds__(kThreads) void zs_embed_join_kernel(const GradParams<T> p) {
    constexpr int V = Chunk<T>::V, W = kThreads / L;
    __shared__ __align__(16) float lds[W][L * V];
    const int64_t block = p.block0 + blockIdx.x, piece = block / p.blocks;
    const int32_t entry = p.leaves[piece];
    if (entry < 0) return;   // of the whole workgroup
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    const int chunk = int(block % p.blocks) * L + l;
    const int chunks = (p.c + V - 1) / V, width = chunks * V;
    int64_t first, last;
    positions(p, first, last);
    int64_t end = p.offsets[int64_t(entry) + 1];
    end = end > last ? last : end;
    int64_t to = (end - 1 - first) / (W * p.len);   // the piece where the run ends
    to = to < piece ? piece : to;
    const int64_t parts = to - piece + 1, each = (parts + W - 1) / W;
    const int64_t i0 = slot * each, i1 = i0 + each < parts ? i0 + each : parts;
    float acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.0f;
    for (int64_t i = i0; i < i1; i += kAhead) {
        float v[kAhead][V];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t at = i + j < i1 ? i + j : i;
            load_sums<V>(p.sums + ((piece + at) * 2 + (at == 0 ? 1 : 0)) * width, chunk, chunks,
                         v[j]);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += i + j < i1 ? v[j][e] : 0.0f;
    }
#pragma unroll
    for (int d = W / 2; d >= 1; d /= 2) {
#pragma unroll
        for (int e = 0; e < V; ++e) lds[slot][l * V + e] = acc[e];
        __syncthreads();
        if (slot + d < W)
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += lds[slot + d][l * V + e];
        __syncthreads();
    }
    if (slot == 0) store_row(p, entry, chunk, acc);
}

// How the positions are cut: lanes of a row, positions in turn.
struct GradPlan {
    int lanes, len, blocks;
    int64_t pieces;
    size_t sums_bytes;
};
GradPlan plan_grad(int64_t n_rows, int64_t c, bool bf16) {
    GradPlan g{};
    const int v = bf16 ? 8 : 4, chunks = int((c + v - 1) / v);
    g.lanes = 1;
    while (g.lanes < 64 && g.lanes < chunks) g.lanes *= 2;
    g.blocks = (chunks + g.lanes - 1) / g.lanes;
    const int w = kThreads / g.lanes;
    g.len = kMaxLen;
    while (g.len > 8 && w * g.len > kMaxPositions) g.len /= 2;
    // shorter turns where there are few workgroups
    while (g.len > 8 && (n_rows + w * g.len - 1) / (w * g.len) * g.blocks < 1024) g.len /= 2;
    const int64_t count = int64_t(w) * g.len;
    g.pieces = (n_rows + count - 1) / count;
    g.sums_bytes = g.pieces > 1 ? (size_t(g.pieces) * 2 * size_t(chunks * v) * 4 + 255) / 256 * 256 : 0;
    return g;
}

template <typename T, int L>
hipError_t run_grad(GradParams<T>& p, hipStream_t stream) {
    constexpr int V = Chunk<T>::V, W = kThreads / L;
    const int chunks = (p.c + V - 1) / V;
    // 16 KiB of zeros a workgroup, at least a row for every L lanes
    const int64_t rows = (16384 / 16) / chunks;
    p.zero_rows = int(rows < W ? W : rows);
    const int64_t zeros = (p.n_entries + p.zero_rows - 1) / p.zero_rows;
    const int64_t work = p.pieces * p.blocks;
    const hipError_t err = launch_ranges(work + zeros, kThreads, [&](int64_t first, int64_t count) {
        p.block0 = first;
        if (p.n_entries <= kFewEntries)
            zs_embed_grad_kernel<T, L, true><<<unsigned(count), kThreads, 0, stream>>>(p);
        else
            zs_embed_grad_kernel<T, L, false><<<unsigned(count), kThreads, 0, stream>>>(p);
        return hipGetLastError();
    });
    if (err != hipSuccess || p.pieces < 2) return err;
    return launch_ranges(work, kThreads, [&](int64_t first, int64_t count) {
        p.block0 = first;
        zs_embed_join_kernel<T, L><<<unsigned(count), kThreads, 0, stream>>>(p);
        return hipGetLastError();
    });
}

template <typename T>
hipError_t embed_grad(const EmbedGradArgs& a, hipStream_t stream) {
    constexpr int V = Chunk<T>::V;
    const GradPlan g = plan_grad(a.n_rows, a.c, sizeof(T) == 2);
    GradParams<T> p{};
    p.gy = static_cast<const T*>(a.gy), p.index = a.index, p.offsets = a.offsets, p.perm = a.perm;
    p.ldg = a.ldg, p.n_rows = a.n_rows, p.n_entries = a.n_entries, p.c = a.c, p.scale = a.scale;
    p.len = g.len, p.blocks = g.blocks, p.pieces = g.pieces;
    p.grad = static_cast<T*>(a.grad);
    p.sums = static_cast<float*>(a.workspace);
    p.leaves = reinterpret_cast<int32_t*>(static_cast<char*>(a.workspace) + g.sums_bytes);
    p.vec = a.c % V == 0 && a.ldg % V == 0 && on16(a.gy) && on16(a.grad);
    switch (g.lanes) {
        case 1: return run_grad<T, 1>(p, stream);
        case 2: return run_grad<T, 2>(p, stream);
        case 4: return run_grad<T, 4>(p, stream);
        case 8: return run_grad<T, 8>(p, stream);
        case 16: return run_grad<T, 16>(p, stream);
        case 32: return run_grad<T, 32>(p, stream);
        default: return run_grad<T, 64>(p, stream);
    }
}

}  // namespace

hipError_t launch_embed(const EmbedArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? embed<__bf16>(a, stream) : embed<float>(a, stream);
}

size_t embed_grad_workspace(int64_t n_rows, int64_t c, bool bf16) {
    const GradPlan g = plan_grad(n_rows, c, bf16);
    return g.sums_bytes ? g.sums_bytes + size_t(g.pieces) * 4 : 0;
}

hipError_t launch_embed_grad(const EmbedGradArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? embed_grad<__bf16>(a, stream) : embed_grad<float>(a, stream);
}

}  // namespace zs
