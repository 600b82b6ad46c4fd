// C ABI of the feed-forward operators (declared in include/sgemm_ffn.h):
// argument checks, workspace and the sequence of kernels of each call.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <initializer_list>

#include "../../include/sgemm_ffn.h"
#include "kernels_ffn.h"
#include "ops_internal.h"

namespace sgemm {
namespace {

constexpr int64_t kMaxFfnSize = int64_t(1) << 26;

bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool type_ok(int type) {
    return type == SGEMM_TYPE_F32 || type == SGEMM_TYPE_F16 || type == SGEMM_TYPE_BF16;
}

// A matrix the call has to read or write: present, aligned to its elements.
bool matrix_ok(const void *p, int type) { return p && aligned(p, type_bytes(type)); }

int64_t at_least_one(int64_t v) { return v > 1 ? v : 1; }

sgemm_status_t status(cudaError_t e) { return e == cudaSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH; }

struct FfnArgs {
    int64_t T, D, F;
    int type, act;
    const void *x;
    int64_t ldx;
    const void *Wg;
    int64_t ldg;
    const void *Wu;
    int64_t ldu;
    const void *Wd;
    int64_t ldd;
};

sgemm_status_t check_ffn(const FfnArgs &a) {
    if (a.T < 0 || a.D < 0 || a.F < 0 || !type_ok(a.type)) return SGEMM_ERR_INVALID_ARG;
    if (a.act != SGEMM_GATE_SILU && a.act != SGEMM_GATE_GELU && a.act != SGEMM_GATE_RELU)
        return SGEMM_ERR_INVALID_ARG;
    if (a.ldx < at_least_one(a.D) || a.ldg < at_least_one(a.F) || a.ldu < at_least_one(a.F) ||
        a.ldd < at_least_one(a.D))
        return SGEMM_ERR_INVALID_ARG;
    if (a.T > kMaxFfnSize || a.D > kMaxFfnSize || a.F > kMaxFfnSize) return SGEMM_ERR_UNSUPPORTED;
    if (a.T > 0 && a.D > 0 && !matrix_ok(a.x, a.type)) return SGEMM_ERR_INVALID_ARG;
    if (a.D > 0 && a.F > 0 &&
        (!matrix_ok(a.Wg, a.type) || !matrix_ok(a.Wu, a.type) || !matrix_ok(a.Wd, a.type)))
        return SGEMM_ERR_INVALID_ARG;
    return SGEMM_OK;
}

int64_t pad8(int64_t v) { return (v + 7) / 8 * 8; }

// Sizes of the pieces of one workspace, then their addresses.
struct Arena {
    size_t bytes = 0;
    char *base = nullptr;
    size_t take(size_t n) {
        const size_t at = bytes;
        bytes += (n + 255) / 256 * 256;
        return at;
    }
    void *at(size_t offset) const { return base + offset; }
};

// A matrix as an operand of the tensor-core products: where it lies, or the
// copy that has to be made of it first.
struct Source {
    FfnOperand op;
    size_t offset = 0;  // of the copy in the workspace
    bool copied = false;
    const void *user = nullptr;
    int64_t ld_user = 0;
};

// The user's rows x cols matrix: read in place where the TMA can (16-bit
// values in 16-byte aligned rows), else through a copy.
Source source(Arena &w, const void *p, int type, int64_t rows, int64_t cols, int64_t ld) {
    Source s;
    s.user = p;
    s.ld_user = ld;
    s.op = FfnOperand{p, rows, cols, ld, rows * ld, 1};
    if (type == kTypeF32 || !aligned(p, 16) || ld % 8 != 0) {
        s.copied = true;
        s.op.ld = pad8(cols);
        s.op.plane_stride = rows * s.op.ld;
        s.op.planes = type == kTypeF32 ? 3 : 1;
        s.offset = w.take((size_t)(s.op.planes * s.op.plane_stride) * 2);
    }
    return s;
}

// An intermediate matrix (h, dg or du) in the workspace, as an operand of the next
// product.  16-bit types: rounded to the type once.  The tensor cores take both
// operands of one type, so 32 bits here would mean two or three planes of it and as
// many products: the rounding adds as much to the outputs' error as their own
// rounding does (against 64 bits, BF16 2.35e-3 of the norm instead of 1.66e-3, FP16
// 2.9e-4 instead of 2.1e-4).  It also has the type's range.
Source intermediate(Arena &w, int type, int64_t rows, int64_t cols) {
    Source s;
    const int planes = type == kTypeF32 ? 3 : 1;
    s.op = FfnOperand{nullptr, rows, cols, pad8(cols), rows * pad8(cols), planes};
    s.offset = w.take((size_t)(planes * s.op.plane_stride) * 2);
    return s;
}

// Where the cut tiles of a product's tail meet; the same for all products of a
// call, which run one after the other.
struct Tail {
    size_t offset = 0;
    float *partials = nullptr;
    int *counters = nullptr;
};
size_t tail_bytes(const OpDevice &dev) {
    return (size_t)2 * dev.num_sms * ffn_slot_floats(false, true) * sizeof(float);
}
// One per tail tile (fewer than workers), CTA of a worker and epilogue warp.
size_t tail_counters(const OpDevice &dev) { return (size_t)dev.num_sms * 8; }

// Takes the workspace (with room for the tail) and gives every piece its
// address.
sgemm_status_t place_all(Arena &w, Tail &tail, const OpDevice &dev, cudaStream_t st,
                         std::initializer_list<Source *> list) {
    tail.offset = w.take(tail_bytes(dev));
    void *base = nullptr;
    sgemm_status_t s = op_workspace(st, w.bytes, &base);
    if (s == SGEMM_OK) s = op_counters(st, tail_counters(dev), &tail.counters);
    if (s != SGEMM_OK) return s;
    w.base = static_cast<char *>(base);
    tail.partials = static_cast<float *>(w.at(tail.offset));
    for (Source *v : list)
        if (v->copied || !v->op.p) v->op.p = w.at(v->offset);
    return SGEMM_OK;
}

sgemm_status_t make_copies(std::initializer_list<const Source *> list, int type,
                           const OpDevice &dev, cudaStream_t st) {
    FfnPrepJob jobs[kFfnPrepJobs];
    int count = 0;
    for (const Source *s : list) {
        if (!s->copied) continue;
        jobs[count++] = FfnPrepJob{s->user, s->ld_user, (int)s->op.rows, (int)s->op.cols,
                                   const_cast<void *>(s->op.p), s->op.ld, s->op.plane_stride};
    }
    return status(launch_ffn_prep(jobs, count, type, dev.num_sms, st));
}

// What the forward pass keeps for the backward pass: u act'(g) and act(g) in
// blocks of 32 x 32 floats, then h as an operand.
struct Kept {
    int64_t keep_cols, block_floats, h_plane;
    int planes;
    int64_t floats() const { return 2 * block_floats + planes * h_plane / 2; }

    Kept(int64_t T, int64_t F, int type) {
        keep_cols = (F + 31) / 32;
        block_floats = (T + 31) / 32 * keep_cols * 1024;
        h_plane = T * pad8(F);
        planes = type == kTypeF32 ? 3 : 1;
    }
    FfnOperand h(float *base, int64_t T, int64_t F) const {
        return FfnOperand{base + 2 * block_floats, T, F, pad8(F), h_plane, planes};
    }
    void set(FfnGemmParams &p, float *base) const {
        p.keep_cols = (int)keep_cols;
        p.keep[0] = base;
        p.keep[1] = base + block_floats;
    }
};

// Single CTAs or pairs, and how the tiles left over after whole rounds are cut
// along k: the least of a model of SM clocks, fitted to GB300 times.  A step (64 k)
// of a 256 x 256 pair tile takes 512, of a 128 x 128 tile 450 (256 of products, but
// its operands pass through shared memory twice in that time; 330 and 560 in its
// place: 64 and 69 us against 60 for the training step 200 x 1000 x 2000).  FP32:
// 1800 of a 256 x 128 pair tile, 2300 of a 128 x 128 one (2048 x 2048 x 8192 step
// 2.20 and 2.67 ms).  Cutting a tile in n pieces costs 128 KB a CTA written (6500
// clocks on all SMs at once) and n times as much read by the last to finish, half
// of both for single CTAs: at 333 x 1000 x 1504 the cut products took 12 us longer
// than their steps.  With FP32 the last to finish also has the longer epilogue (3000
// and 1500 in place of 15000 and 4000: 777 x 1500 x 3000 405 us, so 382).
struct FfnPlan {
    bool pair;
    int workers, long_tiles, extra, full_tiles, tail_tiles, tail_workers;
};

void tile_problems(FfnGemmParams &p, bool pair) {
    const int bm = kFfnBM * (pair ? 2 : 1);
    const int tile_n = ffn_b_cols(p.type == kTypeF32, pair) * (pair ? 2 : 1) / (p.mode == kFfnGate ? 2 : 1);
    p.tiles = 0;
    for (int i = 0; i < p.count; ++i) {
        FfnProblem &q = p.prob[i];
        q.tiles_m = (q.M + bm - 1) / bm;
        q.tiles_n = (q.N + tile_n - 1) / tile_n;
        q.tile0 = p.tiles;
        p.tiles += q.tiles_m * q.tiles_n;
    }
}

FfnPlan ffn_plan(FfnGemmParams &p, int num_sms) {
    FfnPlan best = {};
    double least = -1.0;
    const bool f32 = p.type == kTypeF32;
    bool tall = false;
    for (int i = 0; i < p.count; ++i) tall = tall || p.prob[i].M > kFfnBM;
    auto steps_of = [&](int i) { return (int64_t)p.prob[i].kblocks * p.prob[i].segs; };
    // At most two lengths of tiles: the products up to `others` have the longer.
    int others = 0;
    for (int i = 1; i < p.count; ++i)
        if (steps_of(i) != steps_of(0)) {
            others = i;
            break;
        }
    for (int pair = 0; pair <= (tall ? 1 : 0); ++pair) {
        tile_problems(p, pair != 0);
        FfnPlan q;
        q.pair = pair != 0;
        q.workers = num_sms / (pair ? 2 : 1);
        const int64_t steps = steps_of(p.count - 1);
        const double step = f32 ? (pair ? 1800.0 : 2300.0) : pair ? 512.0 : 450.0;
        const double size = ffn_slot_floats(f32, pair != 0) / 32768.0;
        double whole = 4000.0 + (pair ? 5000.0 : 2500.0);
        q.long_tiles = others ? p.prob[others].tile0 : 0;
        const int more = q.long_tiles % q.workers, fewer = q.workers - more;
        q.extra = 0;
        if (others) {
            // Who has one long tile fewer takes as many others as fit its length.
            const int64_t longer = steps_of(0);
            const int rest = p.tiles - q.long_tiles;
            if (more) q.extra = (int)std::min<int64_t>(longer / steps, rest / fewer);
            whole += step * (double)(q.long_tiles / q.workers * longer + (more ? longer : 0));
        }
        const int rest = p.tiles - q.long_tiles - q.extra * fewer;
        q.full_tiles = rest / q.workers;
        q.tail_tiles = rest % q.workers;
        whole += step * (double)(q.full_tiles * steps);
        // n whole pieces a tile, or (n = 0) even shares for all workers, whose
        // ends meet inside tiles.
        const int most = std::max(1, q.workers / std::max(1, q.tail_tiles));
        for (int n = 0; n <= most; ++n) {
            if (n > steps || (n == 0 && q.tail_tiles * steps < 4 * q.workers)) continue;
            q.tail_workers = n == 1 || q.tail_tiles == 0 ? 0 : n == 0 ? q.workers : q.tail_tiles * n;
            double cost = whole;
            if (n == 1 && q.tail_tiles) cost += step * (double)steps;
            if (q.tail_workers) {
                const double pieces = n == 0 ? (double)q.workers / q.tail_tiles + 1.0 : n;
                cost += step * (double)(q.tail_tiles * steps) / q.tail_workers +
                        size * (f32 ? 15000.0 + 4000.0 * pieces : 8000.0 + 3500.0 * pieces);
            }
            if (least < 0.0 || cost < least) {
                least = cost;
                best = q;
            }
        }
    }
    return best;
}

// A launch of up to kFfnProblems products.  Operands as they lie in memory; a_mn,
// b_mn: their rows run along k.  Those with the longest tiles come first.
struct Launch {
    const OpDevice &dev;
    cudaStream_t st;
    FfnGemmParams p = {};
    FfnMaps maps = {};
    FfnOperand operand[kFfnMaps];
    int operands = 0;

    Launch(const OpDevice &d, cudaStream_t s, const Tail &t, int mode, int type) : dev(d), st(s) {
        p.mode = mode;
        p.type = type;
        p.partials = t.partials;
        p.counters = t.counters;
        p.device = dev.index;
        p.err = dev.err;
        p.timeout_ns = dev.timeout_ns;
        p.skip_loads_from = dev.skip_loads_from;
    }

    FfnProblem &add(int64_t M, int64_t N, int64_t K, const FfnOperand &A, bool a_mn,
                    const FfnOperand &B, bool b_mn, const FfnOperand *A2 = nullptr,
                    const FfnOperand *B2 = nullptr) {
        FfnProblem &q = p.prob[p.count++];
        q.M = (int)M; q.N = (int)N;
        q.segs = A2 ? 2 : 1;
        q.a_mn = a_mn; q.b_mn = b_mn;
        q.kblocks = (int)((K + kFfnBK - 1) / kFfnBK);
        q.a = operands;
        operand[operands++] = A;
        if (A2) operand[operands++] = *A2;
        q.b = operands;
        operand[operands++] = B;
        if (B2) operand[operands++] = *B2;
        return q;
    }

    sgemm_status_t run() {
        int64_t tiles = 0;  // of the smallest kind
        for (int i = 0; i < p.count; ++i)
            tiles += ((int64_t)p.prob[i].M / kFfnBM + 1) * ((int64_t)p.prob[i].N / 64 + 1);
        if (tiles > INT32_MAX / 2) return SGEMM_ERR_UNSUPPORTED;
        const FfnPlan plan = ffn_plan(p, dev.num_sms);
        tile_problems(p, plan.pair);
        p.workers = plan.workers;
        p.long_tiles = plan.long_tiles;
        p.extra = plan.extra;
        p.full_tiles = plan.full_tiles;
        p.tail_tiles = plan.tail_tiles;
        p.tail_workers = plan.tail_workers;
        for (int i = 0; i < p.count; ++i) {
            FfnProblem &q = p.prob[i];
            // Rows of a short A that do not exist are not brought in: what they
            // would add goes into rows of the accumulator that nobody reads.
            const int a_rows = q.a_mn ? kFfnBK : std::min(kFfnBM, (q.M + 7) / 8 * 8);
            const int b_rows = q.b_mn ? kFfnBK : ffn_b_cols(p.type == kTypeF32, plan.pair);
            q.a_bytes = (q.a_mn ? kFfnBM : a_rows) * kFfnBK * 2;
            const int end = i + 1 < p.count ? p.prob[i + 1].a : operands;
            for (int m = q.a; m < end; ++m) {
                const FfnOperand &o = operand[m];
                const sgemm_status_t s =
                    op_encode_16(&maps.m[m], p.type != kTypeF16, o.p, o.rows, o.cols, o.ld, o.planes,
                                 o.plane_stride, m < q.b ? a_rows : b_rows);
                if (s != SGEMM_OK) return s;
            }
        }
        return status(launch_ffn_gemm(maps, p, plan.pair, st));
    }

    void store(FfnProblem &q, void *C, int64_t ld) const {
        q.C[0] = C;
        q.ldc = ld;
        q.c_vec = aligned(C, 16) && ld * type_bytes(p.type) % 16 == 0;
    }
    static void store_planes(FfnProblem &q, const FfnOperand &o) {
        q.C[0] = const_cast<void *>(o.p);
        q.ldc = o.ld;
        q.c_plane = o.plane_stride;
        q.c_vec = 1;
    }
};

// The block's first half: h, and the kept values where `keep` is given.
sgemm_status_t run_gate(const OpDevice &dev, cudaStream_t st, const Tail &tail, const FfnArgs &a,
                        const FfnOperand &x, const FfnOperand &Wg, const FfnOperand &Wu,
                        const FfnOperand &h, const Kept &kept, float *keep) {
    Launch g(dev, st, tail, kFfnGate, a.type);
    g.p.act = a.act;
    Launch::store_planes(g.add(a.T, a.F, a.D, x, false, Wg, true, nullptr, &Wu), h);
    if (keep) kept.set(g.p, keep);
    return g.run();
}

// The whole block for a few rows: one pass over the weights for every eight.
sgemm_status_t run_stream(const OpDevice &dev, cudaStream_t st, const FfnArgs &a, void *y,
                          int64_t ldy) {
    void *h = nullptr;
    const sgemm_status_t s =
        op_workspace(st, (size_t)(std::min<int64_t>(a.T, kFfnStreamRows) * a.F) * sizeof(float), &h);
    if (s != SGEMM_OK) return s;
    const int64_t e = type_bytes(a.type);
    auto vec = [&](const void *p, int64_t ld, int64_t n) {
        return aligned(p, 16) && ld * e % 16 == 0 && n * e % 16 == 0;
    };
    for (int64_t t = 0; t < a.T; t += kFfnStreamRows) {
        FfnStreamParams p = {};
        p.T = (int)std::min<int64_t>(a.T - t, kFfnStreamRows);
        p.N = (int)a.F; p.K = (int)a.D;
        p.act = a.act;
        p.x = static_cast<const char *>(a.x) + t * a.ldx * e; p.ldx = a.ldx;
        p.W = a.Wg; p.ldw = a.ldg;
        p.W2 = a.Wu; p.ldw2 = a.ldu;
        p.y = h; p.ldy = a.F;
        p.device = dev.index;
        if (launch_ffn_stream(p, a.type, true, vec(a.Wg, a.ldg, a.F) && vec(a.Wu, a.ldu, a.F),
                              dev.num_sms, st) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
        p.N = (int)a.D; p.K = (int)a.F;
        p.x = h; p.ldx = a.F;
        p.W = a.Wd; p.ldw = a.ldd;
        p.y = static_cast<char *>(y) + t * ldy * e; p.ldy = ldy;
        if (launch_ffn_stream(p, a.type, false, vec(a.Wd, a.ldd, a.D), dev.num_sms, st) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
    }
    return SGEMM_OK;
}

sgemm_status_t zero_matrix(void *p, int64_t ld, int64_t rows, int64_t cols, int type,
                           cudaStream_t st) {
    const size_t e = type_bytes(type);
    if (!p || rows == 0 || cols == 0) return SGEMM_OK;
    return status(cudaMemset2DAsync(p, ld * e, 0, cols * e, rows, st));
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" {

int64_t sgemm_ffn_saved_floats(int64_t T, int64_t F, int type) {
    if (T < 0 || F < 0 || T > kMaxFfnSize || F > kMaxFfnSize || !type_ok(type)) return 0;
    return T == 0 || F == 0 ? 0 : Kept(T, F, type).floats();
}

sgemm_status_t sgemm_ffn_forward(int64_t T, int64_t D, int64_t F, int type, int activation,
                                 const void *x, int64_t ldx, const void *Wg, int64_t ldg,
                                 const void *Wu, int64_t ldu, const void *Wd, int64_t ldd, void *y,
                                 int64_t ldy, float *saved, void *stream) {
    const FfnArgs a{T, D, F, type, activation, x, ldx, Wg, ldg, Wu, ldu, Wd, ldd};
    sgemm_status_t s = check_ffn(a);
    if (s != SGEMM_OK) return s;
    if (ldy < at_least_one(D) || !aligned(saved, 16)) return SGEMM_ERR_INVALID_ARG;
    if (T == 0 || D == 0) return SGEMM_OK;
    if (!matrix_ok(y, type)) return SGEMM_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    if (F == 0) return zero_matrix(y, ldy, T, D, type, st);
    // Few rows: passes over the weights on the FP32 pipe, one for every eight, cheaper
    // than the tensor cores as long as these would wait for more.  Microseconds of
    // this form and of the tensor cores, weights cold (D x F):
    //   16 bits in place, 4 rows: 1024 x 2048 15, 20; 1280 x 5120 24.5, 23.6; 2048 x
    //     8192 30, 33; 4096 x 12288 59, 69.  8 rows: 512 x 2048 14, 18; 1024 x 4096
    //     20.6, 21.7; 1024 x 6144 26, 24; 1536 x 6144 32, 27; 4096 x 12288 93, 69.
    //   Off 16 bytes (the tensor cores have the weights copied first), 8 rows: 1023 x
    //     4095 27, 33; 2047 x 5461 48, 40; 4095 x 12287 150, 191.  9 rows: 43, 33; 74,
    //     40; 214, 190.
    //   FP32 (split in three first), 24 rows: 1024 x 4096 60, 69; 2048 x 8192 149, 169;
    //     4096 x 12288 308, 438.  25 rows: 72, 69; 186, 168; 403, 439.  Off 16 bytes, 16
    //     rows: 54, 70; 144, 169; 280, 441.  24 rows: 80, 70; 212, 169; 419, 441.
    // So each limit lies where the two cross for some sizes and within a quarter of the
    // faster form for the others.
    const bool in_place = type != kTypeF32 && aligned(Wg, 16) && aligned(Wu, 16) &&
                          aligned(Wd, 16) && ldg % 8 == 0 && ldu % 8 == 0 && ldd % 8 == 0;
    const bool small = D * F <= 6 << 20;
    const int64_t few = type == kTypeF32 ? 24 : in_place && !small ? 4 : 8;
    if (!saved && T <= few) return run_stream(dev, st, a, y, ldy);
    Arena w;
    Tail tail;
    const Kept kept(T, F, type);
    Source vx = source(w, x, type, T, D, ldx), vg = source(w, Wg, type, D, F, ldg),
           vu = source(w, Wu, type, D, F, ldu), vd = source(w, Wd, type, F, D, ldd);
    Source h = intermediate(w, type, T, F);
    s = place_all(w, tail, dev, st, {&vx, &vg, &vu, &vd, &h});
    if (s != SGEMM_OK) return s;
    if (saved) h.op = kept.h(saved, T, F);
    s = make_copies({&vx, &vg, &vu, &vd}, type, dev, st);
    if (s == SGEMM_OK) s = run_gate(dev, st, tail, a, vx.op, vg.op, vu.op, h.op, kept, saved);
    if (s != SGEMM_OK) return s;
    Launch down(dev, st, tail, kFfnStore, type);
    down.store(down.add(T, D, F, h.op, false, vd.op, true), y, ldy);
    return down.run();
}

sgemm_status_t sgemm_ffn_backward(int64_t T, int64_t D, int64_t F, int type, int activation,
                                  const void *x, int64_t ldx, const void *Wg, int64_t ldg,
                                  const void *Wu, int64_t ldu, const void *Wd, int64_t ldd,
                                  const void *dy, int64_t lddy, const float *saved, void *dx,
                                  int64_t lddx, void *dWg, int64_t lddg, void *dWu, int64_t lddu,
                                  void *dWd, int64_t lddd, void *stream) {
    const FfnArgs a{T, D, F, type, activation, x, ldx, Wg, ldg, Wu, ldu, Wd, ldd};
    sgemm_status_t s = check_ffn(a);
    if (s != SGEMM_OK) return s;
    if (lddy < at_least_one(D) || !aligned(saved, 16)) return SGEMM_ERR_INVALID_ARG;
    const bool weights = dWg || dWu || dWd;
    if (dx && (lddx < at_least_one(D) || !aligned(dx, type_bytes(type)))) return SGEMM_ERR_INVALID_ARG;
    if (weights && (lddg < at_least_one(F) || lddu < at_least_one(F) || lddd < at_least_one(D) ||
                    !matrix_ok(dWg, type) || !matrix_ok(dWu, type) || !matrix_ok(dWd, type)))
        return SGEMM_ERR_INVALID_ARG;
    if (D == 0 || (T == 0 && F == 0) || (!dx && !weights)) return SGEMM_OK;
    if (T > 0 && !matrix_ok(dy, type)) return SGEMM_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    if (T == 0 || F == 0) {
        s = zero_matrix(dx, lddx, T, D, type, st);
        if (s == SGEMM_OK && weights) s = zero_matrix(dWg, lddg, D, F, type, st);
        if (s == SGEMM_OK && weights) s = zero_matrix(dWu, lddu, D, F, type, st);
        if (s == SGEMM_OK && weights) s = zero_matrix(dWd, lddd, F, D, type, st);
        return s;
    }
    Arena w;
    Tail tail;
    const Kept kept(T, F, type);
    Source vx = source(w, x, type, T, D, ldx), vg = source(w, Wg, type, D, F, ldg),
           vu = source(w, Wu, type, D, F, ldu), vd = source(w, Wd, type, F, D, ldd),
           vdy = source(w, dy, type, T, D, lddy), dg = intermediate(w, type, T, F),
           du = intermediate(w, type, T, F);
    const size_t kept_at = saved ? 0 : w.take((size_t)kept.floats() * sizeof(float));
    s = place_all(w, tail, dev, st, {&vx, &vg, &vu, &vd, &vdy, &dg, &du});
    if (s != SGEMM_OK) return s;
    float *keep = saved ? const_cast<float *>(saved) : static_cast<float *>(w.at(kept_at));
    const FfnOperand h = kept.h(keep, T, F);
    s = make_copies({&vx, &vg, &vu, &vd, &vdy}, type, dev, st);
    if (s == SGEMM_OK && !saved) s = run_gate(dev, st, tail, a, vx.op, vg.op, vu.op, h, kept, keep);
    if (s != SGEMM_OK) return s;

    Launch grad(dev, st, tail, kFfnGateGrad, type);
    FfnProblem &q = grad.add(T, F, D, vdy.op, false, vd.op, false);
    Launch::store_planes(q, dg.op);
    q.C[1] = const_cast<void *>(du.op.p);
    kept.set(grad.p, keep);
    s = grad.run();
    if (s != SGEMM_OK) return s;
    // The gradients wait for nothing but dg and du: one launch, the longest
    // tiles first (dx sums over 2 F, the weights' over T).
    Launch rest(dev, st, tail, kFfnStore, type);
    const bool dx_first = 2 * ((F + kFfnBK - 1) / kFfnBK) >= (T + kFfnBK - 1) / kFfnBK;
    auto add_dx = [&]() {
        rest.store(rest.add(T, D, F, dg.op, false, vg.op, false, &du.op, &vu.op), dx, lddx);
    };
    if (dx && dx_first) add_dx();
    if (weights) {
        rest.store(rest.add(D, F, T, vx.op, true, dg.op, true), dWg, lddg);
        rest.store(rest.add(D, F, T, vx.op, true, du.op, true), dWu, lddu);
        rest.store(rest.add(F, D, T, h, true, vdy.op, true), dWd, lddd);
    }
    if (dx && !dx_first) add_dx();
    return rest.run();
}

sgemm_status_t sgemm_w4_matvec(int64_t M, int64_t N, int64_t K, int64_t group, int type,
                               const void *x, int64_t ldx, const uint32_t *qweight, int64_t ldq,
                               const void *scales, int64_t lds, const uint8_t *zeros, int64_t ldz,
                               void *y, int64_t ldy, void *stream) {
    if (M < 0 || N < 0 || K < 0 || !type_ok(type) || group < 32 || group % 32 != 0)
        return SGEMM_ERR_INVALID_ARG;
    if (ldx < at_least_one(K) || ldq < at_least_one(N) || lds < at_least_one(N) ||
        ldy < at_least_one(N) || (zeros && ldz < at_least_one(N)))
        return SGEMM_ERR_INVALID_ARG;
    if (N > (int64_t(1) << 30) || K > (int64_t(1) << 30) || M > (int64_t(1) << 20))
        return SGEMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (!matrix_ok(y, type)) return SGEMM_ERR_INVALID_ARG;
    if (K > 0 && (!matrix_ok(x, type) || !matrix_ok(scales, type) || !qweight || !aligned(qweight, 4)))
        return SGEMM_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    const sgemm_status_t s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    const size_t e = type_bytes(type);
    W4Params p = {};
    p.N = (int)N; p.K = (int)K;
    p.group = (int)std::min<int64_t>(group, int64_t(1) << 30);
    p.group_shift = -1;
    for (int b = 5; b < 31; ++b)
        if (p.group == 1 << b) p.group_shift = b;
    p.q = qweight; p.ldq = ldq;
    p.scales = scales; p.lds = lds;
    p.zeros = zeros; p.ldz = ldz;
    p.ldx = ldx; p.ldy = ldy;
    p.x_vec = aligned(x, 16) && (M == 1 || ldx % (16 / (int64_t)e) == 0);
    p.units = (int)((K + kW4UnitK - 1) / kW4UnitK);
    const bool vec = N % 16 == 0 && aligned(qweight, 16) && ldq % 4 == 0 && aligned(scales, 16) &&
                     lds * (int64_t)e % 16 == 0 && (!zeros || (aligned(zeros, 16) && ldz % 16 == 0));
    CUtensorMap map = {};
    if (vec && K > 0) {
        const sgemm_status_t t = op_encode_words(&map, qweight, (K + 7) / 8, N, ldq, kW4BoxCols,
                                                 kW4BoxRows);
        if (t != SGEMM_OK) return t;
    }
    p.device = dev.index;
    p.err = dev.err;
    p.timeout_ns = dev.timeout_ns;
    p.safe_rows = (int)(72 / at_least_one(ldq)) + 1;  // 288 bytes
    const int max_rows = w4_max_rows(type);
    for (int64_t m0 = 0; m0 < M; m0 += max_rows) {
        p.M = (int)std::min<int64_t>(M - m0, max_rows);
        p.x = static_cast<const char *>(x) + m0 * ldx * e;
        p.y = static_cast<char *>(y) + m0 * ldy * e;
        p.warps_n = p.M <= 4 ? 1 : 2;
        // A cluster of CTAs shares K where that shortens the call.  Model, in
        // microseconds, fitted to GB300 times of 11 shapes with one to eight CTAs, of
        // which it takes the best in every one: a wave takes 2.9 and 0.9 for each unit
        // of a warp, an SM 0.028 a unit and 0.24 a CTA.  (8 x 4096 x 12288, bf16: 15.2,
        // 14.5, 12.5, 16.7 us with 1 to 4; 1 x 4096 x 4096: 7.9, 6.0, 6.1, 5.1, and 7.3
        // with 8; 16 x 12288 x 4096: 57, 33, 24, 19, and 16 with 8.)
        const int64_t tiles = (N + kW4Cols * p.warps_n - 1) / (kW4Cols * p.warps_n);
        const int warps_k = kW4Warps / p.warps_n;
        const int parts = type == SGEMM_TYPE_F32 ? 3 : 1;
        // What is left of an SM's places to clusters, which stay inside a group
        // of SMs.
        constexpr double kPlaced[kW4MaxCluster + 1] = {0, 1, 1, .96, .97, .96, .92, .88, .95};
        int cluster = 1;
        double least = 0.0;
        for (int c = 1; c <= kW4MaxCluster && (c == 1 || c * warps_k <= p.units); ++c) {
            const int units = (p.units + c - 1) / c;
            const int staged = std::max(1, std::min(units, kW4StageBytes / w4_unit_bytes(type, p.M)));
            const double places = kPlaced[c] * dev.num_sms * w4_ctas_per_sm(type, p.M, p.group, staged);
            const double waves = ceil(tiles / std::max(1.0, floor(places / c)));
            const double per_warp = (units + warps_k - 1) / warps_k;
            const double cost = waves * (2.87 + 0.92 * per_warp * sqrt((parts * p.M + 7) / 8)) +
                                tiles * (0.0276 * p.warps_n * p.units + 0.24 * c) / dev.num_sms;
            if (c == 1 || cost < least) {
                least = cost;
                cluster = c;
            }
        }
        p.cta_units = (p.units + cluster - 1) / cluster;
        p.chunk_units =
            std::max(1, std::min(p.cta_units, kW4StageBytes / w4_unit_bytes(type, p.M)));
        const cudaError_t err =
            launch_w4(map, p, type, vec, cluster, static_cast<cudaStream_t>(stream));
        if (err != cudaSuccess) return SGEMM_ERR_LAUNCH;
    }
    return SGEMM_OK;
}

sgemm_status_t sgemm_w4_quantize(int64_t N, int64_t K, int64_t group, int type, const void *W,
                                 int64_t ldw, uint32_t *qweight, int64_t ldq, void *scales,
                                 int64_t lds, uint8_t *zeros, int64_t ldz, void *stream) {
    if (N < 0 || K < 0 || !type_ok(type) || group < 32 || group % 32 != 0)
        return SGEMM_ERR_INVALID_ARG;
    if (ldw < at_least_one(N) || ldq < at_least_one(N) || lds < at_least_one(N) ||
        (zeros && ldz < at_least_one(N)))
        return SGEMM_ERR_INVALID_ARG;
    if (N > (int64_t(1) << 30) || K > (int64_t(1) << 30)) return SGEMM_ERR_UNSUPPORTED;
    if (N == 0 || K == 0) return SGEMM_OK;
    if (!matrix_ok(W, type) || !matrix_ok(scales, type) || !qweight || !aligned(qweight, 4))
        return SGEMM_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    const sgemm_status_t s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    W4QuantParams p;
    p.N = (int)N; p.K = (int)K;
    p.group = (int)std::min<int64_t>(group, int64_t(1) << 30);
    p.type = type;
    p.W = W; p.ldw = ldw; p.q = qweight; p.ldq = ldq; p.scales = scales; p.lds = lds;
    p.zeros = zeros; p.ldz = ldz;
    return status(launch_w4_quantize(p, static_cast<cudaStream_t>(stream)));
}

sgemm_status_t sgemm_adamw_step(const sgemm_adamw_tensor_t *tensors, int64_t count, int param_type,
                                int grad_type, int copy_type, int state_bits, double lr,
                                double beta1, double beta2, double eps, double weight_decay,
                                int64_t step, double grad_scale, void *stream) {
    if (count < 0 || (count > 0 && !tensors) || !type_ok(param_type) || !type_ok(grad_type) ||
        !type_ok(copy_type) || (state_bits != 8 && state_bits != 32) || step < 1 ||
        !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0))
        return SGEMM_ERR_INVALID_ARG;
    const size_t state = state_bits == 8 ? 1 : 4;
    for (int64_t i = 0; i < count; ++i) {
        const sgemm_adamw_tensor_t &t = tensors[i];
        if (t.numel < 0) return SGEMM_ERR_INVALID_ARG;
        if (t.numel > (int64_t(1) << 42)) return SGEMM_ERR_UNSUPPORTED;
        if (t.numel == 0) continue;
        if (!matrix_ok(t.param, param_type) || !matrix_ok(t.grad, grad_type) || !t.m || !t.v ||
            !aligned(t.m, state) || !aligned(t.v, state) ||
            (t.copy && !aligned(t.copy, type_bytes(copy_type))))
            return SGEMM_ERR_INVALID_ARG;
        if (state_bits == 8 &&
            (!t.m_scale || !t.v_scale || !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4)))
            return SGEMM_ERR_INVALID_ARG;
    }
    if (count == 0) return SGEMM_OK;
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    const sgemm_status_t s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    const double bc1 = 1.0 - pow(beta1, (double)step), bc2 = 1.0 - pow(beta2, (double)step);
    AdamHyper h;
    h.beta1 = (float)beta1; h.omb1 = (float)(1.0 - beta1);
    h.beta2 = (float)beta2; h.omb2 = (float)(1.0 - beta2);
    h.decay = (float)(1.0 - lr * weight_decay);
    h.step_size = (float)(lr / bc1);
    h.inv_sqrt_bc2 = (float)(1.0 / sqrt(bc2));
    h.eps = (float)eps;
    h.grad_scale = (float)grad_scale;
    h.p_type = param_type; h.g_type = grad_type; h.c_type = copy_type;
    const size_t state_vec = state_bits == 8 ? 8 : 16;
    // Long chunks keep a warp's ring filled; short ones (down to one block per
    // warp) give every SM eight CTAs where there is little to do.
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) total += tensors[i].numel;
    h.chunk = kAdamChunk;
    while (h.chunk > kAdamMinChunk && total / h.chunk < 8 * dev.num_sms) h.chunk /= 2;
    AdamTensor batch[kAdamTensors];
    int n = 0;
    uint64_t chunks = 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    for (int64_t i = 0; i < count; ++i) {
        const sgemm_adamw_tensor_t &t = tensors[i];
        if (t.numel == 0) continue;
        const uint64_t need = (uint64_t)((t.numel + h.chunk - 1) / h.chunk);
        if (n == kAdamTensors || (n > 0 && chunks + need > INT32_MAX)) {
            if (launch_adamw(batch, n, (unsigned)chunks, state_bits, h, dev.index, st) != cudaSuccess)
                return SGEMM_ERR_LAUNCH;
            n = 0;
            chunks = 0;
        }
        AdamTensor &b = batch[n++];
        b.p = t.param; b.g = t.grad; b.m = t.m; b.v = t.v;
        b.ms = t.m_scale; b.vs = t.v_scale; b.copy = t.copy;
        b.numel = t.numel;
        b.chunk0 = (unsigned)chunks;
        b.vec = aligned(t.param, 16) && aligned(t.grad, 16) && aligned(t.m, state_vec) &&
                aligned(t.v, state_vec) && (!t.copy || aligned(t.copy, 16));
        chunks += need;
    }
    return status(n ? launch_adamw(batch, n, (unsigned)chunks, state_bits, h, dev.index, st) : cudaSuccess);
}

}  // extern "C"
