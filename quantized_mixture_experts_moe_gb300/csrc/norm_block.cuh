// Arguments and launch shapes shared by the forward and the backward kernels
// of the block norms (norm_block.cu, norm_block_bwd.cu).
#pragma once

#include "row_ops.cuh"
#include "tc_ptx.cuh"

namespace qmoe {
namespace norm {

constexpr int64_t MAX_COLS = 16384;

inline bool gate_mode_ok(int m) { return m >= QMOE_GATE_NONE && m <= QMOE_GATE_FULL; }

// How the rows of all matrices of a call lie against accesses of `vec` values.
// A row's first value is (base + row * step) % vec values past a boundary; where
// base and step are the same for all matrices, accesses that start that much
// before the row are aligned in each of them, and since a CTA's rows lie a
// multiple of 8 apart, the shift is one for all rows of a CTA.  Odd widths of
// contiguous tensors are of this kind; others go value by value (T=4096, H=4097,
// 16-bit: forward 51 us against 82 value by value, gradient 106 against 332).
struct Lie {
    int vec;
    int64_t cols;
    bool first = true, same = true, whole = cols % 8 == 0;
    int base = 0, step = 0;

    int most() const { return step ? vec - 1 : base; }  // the largest shift of a row
    bool at_zero() const { return whole; }              // all rows begin and end on 16-byte boundaries

    void add(const void* p, int64_t ld, int size) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        const int b = (int)(at / size % vec), s = (int)(ld % vec);
        if (first) {
            base = b;
            step = s;
            first = false;
        }
        same = same && base == b && step == s;
        whole = whole && aligned16(p) && ld * size % 16 == 0;
    }
};

// How a row is cut: nv vectors of vec columns in each of `threads` threads, at
// least `values` each, then 16 and 32 where that takes more than 512 threads;
// rows of 32 threads go four to a CTA.
struct Shape {
    int vec, nv, threads, rows_per_cta;
    int values() const { return vec * nv; }
};

// vec: the columns of one access (8 where all matrices are 16-bit; 4 beside an
// fp32 one, so that its lanes' 16 bytes touch; 1 for rows off the 16-byte
// boundaries).
template <typename RT, typename YT>
constexpr int wide_vec() { return sizeof(RT) == 4 || sizeof(YT) == 4 ? 4 : 8; }

inline Shape shape_for(int64_t cols, int vec, int values) {
    Shape s;
    s.vec = vec;
    for (;; values *= 2) {
        s.nv = values / s.vec;
        const int64_t per = (cols + values - 1) / values;
        s.threads = (int)((per + 31) / 32 * 32);
        if (s.threads <= 512 || values == 32) break;
    }
    s.rows_per_cta = s.threads == 32 ? 4 : 1;
    return s;
}
// With room for a shift where the width is off the access, as long as that takes
// no more values a thread, nor (`exact`) more threads.
inline Shape shape_of(int64_t cols, int vec, int values, bool exact) {
    const Shape s = shape_for(cols, vec, values);
    if (cols % vec == 0) return s;
    const Shape r = shape_for(cols + vec - 1, vec, values);
    return r.threads <= 512 && r.nv == s.nv && (!exact || r.threads == s.threads) ? r : s;
}
// Whether rows of any shift of `lie` end within the threads' columns.
inline bool fits(const Shape& s, const Lie& lie) {
    return lie.same && lie.cols + lie.most() <= (int64_t)s.values() * s.threads;
}

// ------------------------------------------------------------------ rows on their way
//
// The next rows come by bulk copies into a ring of shared memory stages while
// the present one is worked on: HBM wants some 40 KB in flight for each SM,
// more than the registers of the threads that share a row can hold beside
// their work, and one thread's bulk copies cost the others no instructions
// (with a cp.async by each thread for its own values the kernels were bound by
// instruction issue).  Rows that do not start on 16-byte boundaries are copied
// by the 16-byte granules that they lie in.  A granule reaches past its row;
// before the first row and after the last one values are copied one by one
// instead.  (Rows narrower than a granule may still share one with what lies
// before or after the matrix: it is read, in the same 16 bytes, and not used.)

// One matrix that a kernel reads: rows of `cols` values, at `off` in a stage.
struct Source {
    const void* p;  // null: not given
    int64_t ld;
    int off;
};

constexpr int MAX_STAGES = 6, MAX_ROWS = 4;  // stages of a ring, rings of a CTA

constexpr int stage_bytes(int64_t cols, int size) { return (int)((cols * size + 15) / 16 * 16 + 16); }

// Stages that fit in a CTA's share of an SM's shared memory, of which the system
// keeps 1 KB a CTA and the kernels' own arrays take less than half of one.
constexpr int64_t room_of(int64_t other_bytes, int ctas_per_sm) { return 226 * 1024 / ctas_per_sm - 1536 - other_bytes; }
inline int stages_of(int64_t bytes_per_stage, int64_t other_bytes, int ctas_per_sm) {
    const int64_t n = room_of(other_bytes, ctas_per_sm) / bytes_per_stage;
    return n > MAX_STAGES ? MAX_STAGES : n > 0 ? (int)n : 0;
}

// One thread's part in filling the ring: the rows of one matrix.
struct Feed {
    const uint8_t* p = nullptr;  // the next row to send for (null: this thread has no matrix)
    int64_t step = 0;            // bytes from one row of this ring to the next
    int off = 0, bytes = 0;      // its place in a stage; the bytes of a row

    __device__ __forceinline__ void take(const Source& s, int size, int& turn, int id, int64_t row, int64_t stride,
                                         int cols) {
        if (!s.p) return;
        if (turn++ == id) {
            p = static_cast<const uint8_t*>(s.p) + row * s.ld * size;
            step = stride * s.ld * size;
            off = s.off;
            bytes = cols * size;
        }
    }
    // Sends for row `row` of `rows` and tells the barrier.  WHOLE: rows on 16-byte boundaries.
    template <bool WHOLE>
    __device__ __forceinline__ void send(uint8_t* stage, int64_t row, int64_t rows, uint64_t* bar) {
        uint8_t* dst = stage + off;
        if constexpr (WHOLE) {
            tc::mbar_arrive_expect_tx(bar, bytes);
            tc::bulk_load(dst, p, bytes, bar);
        } else {
            const uintptr_t g0 = reinterpret_cast<uintptr_t>(p), g1 = g0 + (uintptr_t)bytes;
            const uintptr_t base = g0 & ~uintptr_t(15);
            uintptr_t a0 = base, a1 = (g1 + 15) & ~uintptr_t(15);
            if (row == 0 && a0 < g0) a0 += 16;
            if (row == rows - 1 && a1 > g1) a1 -= 16;
            if (a1 < a0) a1 = a0;  // a row within one granule
            auto one_by_one = [&](uintptr_t b, uintptr_t e) {
                for (; b < e; b += 2)  // values are 2 or 4 bytes, aligned
                    *reinterpret_cast<uint16_t*>(dst + (b - base)) = *reinterpret_cast<const uint16_t*>(b);
            };
            if (a0 > g0) one_by_one(g0, a0 < g1 ? a0 : g1);
            if (a1 < g1) one_by_one(a1 > g0 ? a1 : g0, g1);
            tc::mbar_arrive_expect_tx(bar, (uint32_t)(a1 - a0));
            if (a1 > a0) tc::bulk_load(dst + (a0 - base), reinterpret_cast<const void*>(a0), (uint32_t)(a1 - a0), bar);
        }
        p += step;
    }
};

// How a kernel reads a row: by accesses of VEC columns.  Without SHIFT all rows
// begin and end on an access's boundaries; with it they begin `shift` columns past
// one, so that a row's first and last access reach past it.  (A kernel that
// keeps both cases open spends 5 to 20% more on the first: H=4096 forward 28 us
// for 26, gradient 70 for 59.)
// A thread's columns.
template <int VEC, bool SHIFT>
struct Columns {
    int cols, shift;
    bool fp32;  // fp32 values for each column may be read VEC at a time (16-byte boundaries, no shift)

    // first column of the thread's v-th access
    __device__ __forceinline__ int at(int v) const {
        return (int)(v * blockDim.x + threadIdx.x) * VEC - (SHIFT ? shift : 0);
    }
    __device__ __forceinline__ bool live(int c) const { return c < cols && (!SHIFT || c > -VEC); }
    __device__ __forceinline__ bool whole(int c) const { return !SHIFT || (c >= 0 && c + VEC <= cols); }
    __device__ __forceinline__ bool in(int c) const { return !SHIFT || (c >= 0 && c < cols); }
};

// Zeros for an access's columns outside the row.
template <int VEC, bool SHIFT>
__device__ __forceinline__ void clear_outside(const Columns<VEC, SHIFT>& k, int c, float* v) {
    if constexpr (SHIFT) {
        if (k.whole(c)) return;
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = k.in(c + i) ? v[i] : 0.f;
    }
}
// fp32 values of the columns of an access (weights), 0 outside the row.
template <int VEC, bool SHIFT>
__device__ __forceinline__ void load_columns(const Columns<VEC, SHIFT>& k, const float* w, int c, float* v) {
    if (!SHIFT || (k.fp32 && k.whole(c))) {
        row::load<VEC>(w + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = k.in(c + i) ? w[c + i] : 0.f;
    }
}
// VEC values of a row of a matrix.
template <int VEC, bool SHIFT, typename T>
__device__ __forceinline__ void store_columns(const Columns<VEC, SHIFT>& k, T* dst, int c, const float* v) {
    if (k.whole(c)) {
        row::store<VEC>(dst + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (k.in(c + i)) dst[c + i] = row::from_f32<T>(v[i]);
    }
}

// One access of a row, widened; zeros outside it.  RING: the row lies in a
// stage, whose granules reach past it; else straight from the matrix.
template <bool RING, int VEC, bool SHIFT, typename T>
__device__ __forceinline__ void read_columns(const Columns<VEC, SHIFT>& k, const T* src, int c, float* v) {
    if (RING || k.whole(c)) {
        row::load<VEC>(src + c, v);
        clear_outside(k, c, v);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = k.in(c + i) ? row::to_f32(src[c + i]) : 0.f;
    }
}
template <bool RING, typename T, int VEC, bool SHIFT>
__device__ __forceinline__ const T* row_at(const Columns<VEC, SHIFT>&, const Source& s, const uint8_t* stage,
                                           int64_t row) {
    if (RING && VEC > 1 && !SHIFT) return reinterpret_cast<const T*>(stage + s.off);
    const T* src = static_cast<const T*>(s.p) + row * s.ld;
    return RING ? reinterpret_cast<const T*>(stage + s.off + (reinterpret_cast<uintptr_t>(src) & 15)) : src;
}
// This thread's values of a row.
template <int NV, bool RING, typename T, int VEC, bool SHIFT>
__device__ __forceinline__ void read_row(const Source& s, const uint8_t* stage, int64_t row,
                                         const Columns<VEC, SHIFT>& k, float* v) {
    const T* src = row_at<RING, T>(k, s, stage, row);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = k.at(i);
        if (k.live(c)) {
            read_columns<RING>(k, src, c, &v[i * VEC]);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[i * VEC + j] = 0.f;
        }
    }
}

// The ring of one row's threads.  Its first threads send, each for the rows of
// one matrix (one thread that sent for all of them took 1,100 cycles a row, and
// the others waited for it at the row's next barrier).  A stage is refilled
// when its row's threads have met once more after reading it.
template <bool WHOLE>
struct Ring {
    uint64_t* full;
    uint8_t* base;
    int stages, bytes;
    int64_t rows, stride;
    Feed feed;
    int stage = 0;
    uint32_t phase = 0;
    // a copy did not arrive in time: what follows is NaN, and no more is sent for (what had been, before that wait, has
    // had the wait's 2 s to land)
    bool lost = false;

    __device__ __forceinline__ void post(int64_t row, int at) {
        if (feed.p && row < rows) feed.template send<WHOLE>(base + at * bytes, row, rows, &full[at]);
    }
    __device__ __forceinline__ void begin(int64_t row) {
        for (int i = 0; i + 1 < stages || i == 0; ++i) post(row + i * stride, i);
    }
    // The stage of the present row.  One lane of a warp waits (32 lanes that ask the same barrier are served one by
    // one); __syncwarp passes on to the others what it guards.
    __device__ __forceinline__ const uint8_t* wait() {
        int late = 0;
        if ((threadIdx.x & 31) == 0 && !lost) late = !tc::mbar_wait(&full[stage], phase);
        if (__shfl_sync(0xFFFFFFFFu, late, 0)) {
            lost = true;
            feed.p = nullptr;
        }
        __syncwarp();
        return base + stage * bytes;
    }
    // The row's threads have met since `row` was waited for: the stage read before it is free.
    __device__ __forceinline__ void refill(int64_t row) {
        if (stages > 1) post(row + (stages - 1) * stride, stage == 0 ? stages - 1 : stage - 1);
    }
    __device__ __forceinline__ void next() {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    }
};

// The threads of a row meet.
__device__ __forceinline__ void row_barrier() {
    if (blockDim.x == 32) __syncwarp();
    else __syncthreads();
}

// (stream type, block type): the same type twice, or a 16-bit block beside an
// fp32 stream.
template <template <typename, typename> class F, typename... A>
inline int by_types(int rt, int yt, A&&... a) {
    if (rt == QMOE_F32 && yt == QMOE_F32) return F<float, float>::go(a...);
    if (rt == QMOE_F32 && yt == QMOE_BF16) return F<float, __nv_bfloat16>::go(a...);
    if (rt == QMOE_F32 && yt == QMOE_F16) return F<float, __half>::go(a...);
    if (rt == QMOE_BF16 && yt == QMOE_BF16) return F<__nv_bfloat16, __nv_bfloat16>::go(a...);
    if (rt == QMOE_F16 && yt == QMOE_F16) return F<__half, __half>::go(a...);
    return QMOE_ERR_ARG;
}

inline bool types_ok(int rt, int yt) {
    return row::dtype_ok(rt) && row::dtype_ok(yt) && (rt == yt || rt == QMOE_F32);
}

}  // namespace norm
}  // namespace qmoe
