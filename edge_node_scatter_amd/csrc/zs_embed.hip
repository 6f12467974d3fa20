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
template <typename T, int L, int U>
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
                                   : load_chunk(p.table + from[u] * p.ldt, chunk, p.c, p.vec);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = base + u * kRows + slot;
                if (row >= p.n_rows) continue;
                float f[V];
                Chunk<T>::unpack(v[u], f);
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] *= p.scale;
                // a row of no entry is +0 whatever the scale's sign
                store_any(p.y + row * p.c, chunk, p.c, p.vec,
                          from[u] < 0 ? v[u] : Chunk<T>::pack(f));
            }
        }
    }
}

template <typename T, int L>
hipError_t run_embed(const EmbedParams<T>& p, hipStream_t stream) {
    constexpr int kRows = 256 / L;
    const int64_t one = (p.n_rows + kRows - 1) / kRows;
    // four rows at a time where that still leaves several workgroups for every unit
    if (one >= 4096) {
        const int64_t want = (one + 3) / 4;
        zs_embed_kernel<T, L, 4><<<unsigned(want < 1 << 20 ? want : 1 << 20), 256, 0, stream>>>(p);
    } else {
        zs_embed_kernel<T, L, 1><<<unsigned(one), 256, 0, stream>>>(p);
    }
    return hipGetLastError();
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
    float* sums;      // [pieces][2][c]: of the run that enters a piece, of the one that leaves it
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
// fp32 sums of a chunk's columns.
template <int V>
__device__ inline void store_sums(float* row, int chunk, int c, const float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (chunk * V + i < c) row[chunk * V + i] = v[i];
}

template <typename T, int L>
__global__ __launch_bounds__(kThreads) void zs_embed_grad_kernel(const GradParams<T> p) {
    constexpr int V = Chunk<T>::V, W = kThreads / L;
    __shared__ int32_t rows[kMaxPositions];
    __shared__ int32_t entry_of[kMaxPositions + 2];   // one position before and behind
    __shared__ float head[W][L * V], tail[W][L * V];
    __shared__ int32_t tail_entry[W];
    __shared__ bool has_head[W], through[W];
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    const int chunks = (p.c + V - 1) / V;
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
    for (int i = int(threadIdx.x) - 1; i <= count; i += kThreads) {
        const int64_t q = q0 + i;
        int64_t row = -1, v = -1;
        if (q >= first && q < last) {
            row = p.perm ? p.perm[q] : q;
            if (row >= 0 && row < p.n_rows) v = p.index[row];
            if (v < 0 || v >= p.n_entries) v = -1;
        }
        entry_of[i + 1] = int32_t(v);
        if (i >= 0 && i < count) rows[i] = int32_t(row);
    }
    __syncthreads();
    const int i0 = slot * p.len, i1 = i0 + p.len;
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.0f;
    int32_t cur = entry_of[i0 + 1];
    bool entered = cur >= 0 && cur == entry_of[i0];
    bool head_done = false;
    for (int i = i0; i < i1; i += kAhead) {
        u32x4 raw[kAhead];
        int32_t at[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            at[j] = i + j < i1 ? entry_of[i + j + 1] : -1;
            raw[j] = at[j] < 0 ? u32x4{0, 0, 0, 0}
                               : load_chunk(p.gy + int64_t(rows[i + j]) * p.ldg, chunk, p.c, p.vec);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (i + j >= i1) break;
            if (at[j] != cur) {   // a run ends here
                if (entered) {
#pragma unroll
                    for (int e = 0; e < V; ++e) head[slot][l * V + e] = acc[e];
                    head_done = true;
                } else if (cur >= 0) {
                    store_row(p, cur, chunk, acc);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] = 0.0f;
                cur = at[j];
                entered = false;
            }
            float f[V];
            Chunk<T>::unpack(raw[j], f);
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += f[e];
        }
    }
    const bool goes_on = cur >= 0 && cur == entry_of[i1 + 1];
    bool starts = false;   // a run starts among these positions and goes on
    if (entered) {
#pragma unroll
        for (int e = 0; e < V; ++e) head[slot][l * V + e] = acc[e];
        head_done = true;
    } else if (goes_on) {
#pragma unroll
        for (int e = 0; e < V; ++e) tail[slot][l * V + e] = acc[e];
        starts = true;
    } else if (cur >= 0) {
        store_row(p, cur, chunk, acc);
    }
    if (l == 0) {
        tail_entry[slot] = starts ? cur : -1;
        has_head[slot] = head_done;
        through[slot] = entered && goes_on;
    }
    __syncthreads();
    // runs that enter the workgroup's positions, by the first lanes, and runs that start
    // in these lanes' positions
    for (int pass = 0; pass < 2; ++pass) {
        int s = slot;
        bool leaves;
        if (pass == 0) {
            if (slot != 0 || !has_head[0]) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = head[0][l * V + e];
            leaves = through[0];
        } else {
            if (!starts) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = tail[slot][l * V + e];
            leaves = true;
        }
        while (leaves && s + 1 < W && has_head[s + 1]) {
            ++s;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += head[s][l * V + e];
            leaves = through[s];
        }
        if (pass == 0)
            store_sums<V>(p.sums + piece * 2 * p.c, chunk, p.c, acc);
        else if (leaves)
            store_sums<V>(p.sums + (piece * 2 + 1) * p.c, chunk, p.c, acc);
        else
            store_row(p, tail_entry[slot], chunk, acc);
        if (pass == 1 && leaves && l == 0 && p.pieces > 1) p.leaves[piece] = tail_entry[slot];
    }
    // no run leaves: the last lanes know (the only ones whose run can)
    if (threadIdx.x == kThreads - 1 && p.pieces > 1) {
        int s = W - 1;
        while (s > 0 && through[s]) --s;
        if (!(through[s] || tail_entry[s] >= 0) || (s == 0 && through[0]))
            p.leaves[piece] = -1;
    }
}

// Adds the sums of a run that goes over several pieces, in order: L lanes a row and
// W parts, joined in LDS.
template <typename T, int L>
__global__ __launch_bounds__(kThreads) void zs_embed_join_kernel(const GradParams<T> p) {
    constexpr int V = Chunk<T>::V, W = kThreads / L;
    __shared__ float lds[W][L * V];
    const int64_t block = p.block0 + blockIdx.x, piece = block / p.blocks;
    const int32_t entry = p.leaves[piece];
    if (entry < 0) return;   // of the whole workgroup
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    const int chunk = int(block % p.blocks) * L + l;
    int64_t first, last;
    positions(p, first, last);
    int64_t end = p.offsets[int64_t(entry) + 1];
    end = end > last ? last : end;
    int64_t to = (end - 1 - first) / (W * p.len);   // the piece where the run ends
    to = to < piece ? piece : to;
    const int64_t parts = to - piece + 1, each = (parts + W - 1) / W;
    float acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.0f;
    for (int64_t i = slot * each; i < (slot + 1) * each && i < parts; ++i) {
        const float* row = p.sums + ((piece + i) * 2 + (i == 0 ? 1 : 0)) * p.c;
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (chunk * V + e < p.c) acc[e] += row[chunk * V + e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) lds[slot][l * V + e] = acc[e];
    __syncthreads();
    if (slot != 0) return;
    for (int s = 1; s < W && s * each < parts; ++s)
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += lds[s][l * V + e];
    if (chunk * V < p.c) store_row(p, entry, chunk, acc);
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
    g.sums_bytes = g.pieces > 1 ? (size_t(g.pieces) * 2 * size_t(c) * 4 + 255) / 256 * 256 : 0;
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
        zs_embed_grad_kernel<T, L><<<unsigned(count), kThreads, 0, stream>>>(p);
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
