// Weight updates of the C ABI (declared in include/wgrad.h): the orthogonalised
// update and the embedding table's lookup and gradient.  Validation, workspace
// layout and launches; no device memory is allocated here.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <string>

#include "../../include/wgrad.h"
#include "host.h"
#include "k_embedding.cuh"
#include "k_muon_gemm.cuh"

namespace wg {

cudaError_t read_update_status(unsigned int* v) { return cudaMemcpyFromSymbol(v, g_status, sizeof *v); }
cudaError_t write_update_status(unsigned int v) { return cudaMemcpyToSymbol(g_status, &v, sizeof v); }

}  // namespace wg

namespace {

using wg::aligned16;
using wg::cuda_fail;
using wg::num_sms;
using wg::set_err;

int esize(int dtype) { return dtype == WG_FP32 ? 4 : 2; }
bool dtype_ok(int d) { return d == WG_FP32 || d == WG_BF16 || d == WG_FP16; }
bool aligned_to(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0; }

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

template <typename... P, typename... A>
int launch(const char* what, void (*k)(P...), dim3 grid, dim3 block, int smem, cudaStream_t stream, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    unsigned na = 0;
    wg::pdl_config(&cfg, attr, &na, stream);
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = (size_t)smem;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k, args...);
    return e == cudaSuccess ? WG_OK : cuda_fail(what, e);
}

int check_workspace(size_t need, const void* workspace, size_t ws_bytes)
{
    if (need == 0) return WG_OK;
    if (!workspace || ws_bytes < need) {
        char buf[160];
        snprintf(buf, sizeof buf, "workspace of %zu bytes needed (got %zu%s)", need, ws_bytes, workspace ? "" : ", NULL");
        return set_err(WG_ERR_WORKSPACE, buf);
    }
    if (!aligned16(workspace)) return set_err(WG_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    return WG_OK;
}

// ---------------------------------------------------------------- orthogonalised update
// Elements that a layout may span: their bytes and the sums of their addresses stay in 64 bits.
constexpr long long kMaxSpan = 1LL << 48;

constexpr int kMuonMaxDim = 32768, kMuonMaxSteps = 16, kMuonMaxParts = 1216;

struct MuonPlan {
    wg_muon_problem p;
    float coef[kMuonMaxSteps][3];
    bool gram;            // the Gram-matrix kernel
    wg::GramParams g;     // its problem (pointers are set by the call), with every launch's steps
    int launches, first[kMuonMaxSteps + 1];  // its launches, and the first step of each (and the end)
    int P, blocks;        // rows of a block of the Gram matrix, blocks
    int ldx, m, ldm, nparts;
    int pairs;
    bool two;             // general form: A, B and X of the products have two fp16 values
    size_t off_x[2], off_xlo[2], off_a, off_b, off_alo, off_blo, off_part, off_sums, off_arrived, bytes;
};

// CTAs of the Gram-matrix kernel's largest cluster: 16 where the device takes it
// (beyond the portable 8), asked once per device.
int muon_gram_max_cluster()
{
    static std::mutex mu;
    static std::map<int, int> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 16;
    }
    std::lock_guard<std::mutex> lk(mu);
    auto it = cache.find(dev);
    if (it != cache.end()) return it->second;
    int n = 0;
    const int smem = wg::gram_smem_bytes(128);
    if (wg::ensure_smem(wg::muon_gram_kernel<128, true>, smem) == WG_OK &&
        cudaFuncSetAttribute(wg::muon_gram_kernel<128, true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 16;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr, cfg.numAttrs = 1;
        cfg.gridDim = dim3(16), cfg.blockDim = dim3(wg::kGramBlock);
        cfg.dynamicSmemBytes = (size_t)smem;
        if (cudaOccupancyMaxActiveClusters(&n, wg::muon_gram_kernel<128, true>, &cfg) != cudaSuccess) n = 0;
    }
    cudaGetLastError();
    return cache[dev] = n > 0 ? 16 : 8;
}

// MMAs add to their sums with truncation: a sum of equal signs over 16 n elements comes
// out short by 0.95e-7 n^2 / (n + 5) of itself, measured on products of matrices of rank
// one: 1.8e-7 for n = 4, 4.5e-7 for 8, 12e-7 for 16, 59e-7 for 64 and 509e-7 for 512.
// Maps with slopes of 1e4 and more make that visible (the factors that fall from 8.3
// have 3e4 at 1: 256 x 512 of rank one 4.8e-2 off without, 3e-3 with), so it is put
// back; sums of mixed signs lose less, and no map makes much of theirs.
double muon_put_back(double n) { return 1.0 + 0.95e-7 * n * n / (n + 5.0); }


// Largest value over s in [0, smax] of what a step (a, b, c) makes of a singular value s,
// and of the factor that it multiplies s by.
void factor_range(const float* k, double smax, double* grown, double* factor)
{
    *grown = *factor = 0.0;
    for (int i = 0; i <= 512; ++i) {
        const double s = smax * i / 512, l = s * s, v = fabs(k[0] + k[1] * l + k[2] * l * l);
        *grown = std::max(*grown, s * v);
        *factor = std::max(*factor, v);
    }
}

// The Gram-matrix kernel's problem: blocks of whole matrices, CTAs of a cluster,
// and the powers of two that bring each operand's largest singular value to at
// most 2^13 in fp16 (a factor of eight is left to roundings).
void muon_gram_plan(MuonPlan* pl)
{
    const wg_muon_problem& q = pl->p;
    wg::GramParams& g = pl->g;
    g = wg::GramParams();
    pl->P = pl->m <= 64 ? 64 : 128;
    g.N = std::max(q.rows, q.cols);
    g.F = std::min(pl->P / pl->m, q.batch);
    g.wide = q.rows <= q.cols;
    g.chunks = (g.N + 63) / 64;
    g.steps = q.steps;
    pl->blocks = (q.batch + g.F - 1) / g.F;
    // A CTA per chunk up to the largest cluster, while every block has its cluster at
    // once (96 x 3456: 44 us with 16 CTAs, 57 with 8, 90 with 4).
    g.C = 1;
    const int cmax = muon_gram_max_cluster();
    while (g.C < cmax && 2 * g.C <= g.chunks && 2LL * g.C * pl->blocks <= num_sms()) g.C *= 2;
    g.kn = (g.F * pl->m + 15) / 16;
    // Steps of a launch.  An error of A or Q in directions that u (nearly) lacks grows with
    // the product of the steps' factors |a + b l + c l^2|, A's with its square.  The largest
    // error of X in a simulation of every rounding, over spectra of one direction and noise
    // of many sizes, for 3 x 7 (the worst) and 64 x 576: products of up to 600 in a launch
    // (five default steps) 1.7e-3 and 3e-4, up to 170 (four) 1e-4 and 2e-5, 1,700 (six)
    // 2e-2 and 3e-3, 5,800 (seven) 0.2 and 4e-2; beyond, A leaves [0, 1] and X is NaN.  So
    // one launch up to 600, and where that is not enough launches of up to 170, with which
    // six and seven steps are 1.2e-3 off at most (5e-4 for 64 x 576).
    double factor[kMuonMaxSteps], all = 1.0, smax = 1.0;
    for (int k = 0; k < q.steps; ++k) {
        double grown;
        factor_range(pl->coef[k], smax, &grown, &factor[k]);
        all *= std::max(factor[k], 1.0);
        smax = std::max(grown, 1e-3);
    }
    pl->launches = 1, pl->first[0] = 0;
    double part = 1.0;
    for (int k = 0; k < q.steps; ++k) {
        const double f = std::max(factor[k], 1.0);
        if (all > 600.0 && k > 0 && part * f > 170.0) pl->first[pl->launches++] = k, part = 1.0;
        part *= f;
    }
    pl->first[pl->launches] = q.steps;
    auto power = [](double bound) { return ldexpf(1.f, (int)floor(log2(8192.0 / std::max(bound, 1e-6)))); };
    const double put_back = muon_put_back(pl->m / 16.0);
    smax = 1.0;
    for (int n = 0; n < pl->launches; ++n) {
        double grid[513], prod[513];
        for (int i = 0; i <= 512; ++i) grid[i] = smax * i / 512, prod[i] = 1.0;
        float ra = 1.f;  // A = ra * (its sums in tensor memory)
        for (int k = pl->first[n]; k < pl->first[n + 1]; ++k) {
            const float* c = pl->coef[k];
            wg::GramParams::Step& w = g.step[k];
            double pmax = 0.0, spmax = 0.0, grown = 0.0, qmax = 0.0;
            for (int i = 0; i <= 512; ++i) {
                const double s = smax * i / 512, l = s * s, v = c[0] + c[1] * l + c[2] * l * l;
                pmax = std::max(pmax, fabs(v)), spmax = std::max(spmax, l * fabs(v)), grown = std::max(grown, s * fabs(v));
                const double t = grid[i] * grid[i], u = c[0] + c[1] * t + c[2] * t * t;
                prod[i] *= u, grid[i] *= u;
                qmax = std::max(qmax, fabs(prod[i]));
            }
            w.sa = power(smax * smax), w.sp = power(pmax), w.ss = power(spmax), w.sq = power(qmax);
            w.pa = c[0], w.pb = c[1] * ra, w.pc = (float)(c[2] / (w.sa * w.sa) * put_back);
            w.rs = (float)(put_back / (w.sa * w.sp));
            w.rq = k > pl->first[n] ? (float)(put_back / (w.sp * g.step[k - 1].sq)) : 1.f;
            w.ra = ra = (float)(put_back / (w.ss * w.sp));
            smax = std::max(grown, 1e-3);
        }
    }
}

// Largest value over s in [0, smax] of what a step (a, b, c) makes of a singular
// value s, and of |b s^2 + c s^4|, on a grid fine enough for a quintic.
void step_range(const float* k, double smax, double* grown, double* poly)
{
    *grown = *poly = 0.0;
    for (int i = 0; i <= 4096; ++i) {
        const double s = smax * i / 4096, l = s * s, q = k[1] * l + k[2] * l * l;
        *grown = std::max(*grown, fabs(s * (k[0] + q)));
        *poly = std::max(*poly, fabs(q));
    }
}

// What rounding A, B and X to 11 bits costs the general form, in units of 2^-15 or so:
// the largest |b| s^3 + |c| s^5 of a step, grown by the slopes of the later steps' maps,
// over s in [0, 1] and all steps.  Five default steps have 88, six 144, seven 231; an
// error of X of 3.0e-3, 4.4e-3 and 4.8e-3 (the largest over spectra, 130 x 160 to 256 x
// 512, simulated).  Factors that fall from 8.3 have 1e5: rank one was 18 to 45% off, and
// with three cubic steps behind them 170 times too large.
double muon_single_error(const float (*coef)[3], int steps)
{
    double worst = 0.0;
    for (int i = 0; i <= 4096; ++i) {
        double s = i / 4096.0, e = 0.0;
        for (int k = 0; k < steps; ++k) {
            const double a = coef[k][0], b = coef[k][1], c = coef[k][2], l = s * s;
            e = e * fabs(a + 3.0 * b * l + 5.0 * c * l * l) + (fabs(b) * l + fabs(c) * l * l) * s;
            worst = std::max(worst, e);
            s *= a + b * l + c * l * l;
        }
    }
    return worst;
}

bool muon_factors_ok(const wg_muon_problem& p)
{
    return p.mu >= 0.f && p.mu < 1.f && p.dampening >= 0.f && p.dampening <= 1.f && p.eps >= 0.f && isfinite(p.eps) &&
           isfinite(p.scale) && isfinite(p.lr) && isfinite(p.weight_decay);
}

int make_muon_plan(const wg_muon_problem* p, MuonPlan* pl)
{
    if (!p) return set_err(WG_ERR_INVALID_ARGUMENT, "problem is NULL");
    if (p->batch < 1 || p->rows < 1 || p->cols < 1)
        return set_err(WG_ERR_INVALID_ARGUMENT, "batch, rows and cols must be at least 1");
    if (p->rows > kMuonMaxDim || p->cols > kMuonMaxDim || p->batch > 65535)
        return set_err(WG_ERR_NOT_SUPPORTED, "rows and cols up to 32768 and batch up to 65535 are supported");
    if (!dtype_ok(p->grad_dtype) || !dtype_ok(p->out_dtype) || !dtype_ok(p->weight_dtype))
        return set_err(WG_ERR_INVALID_ARGUMENT, "grad_dtype, out_dtype and weight_dtype must be WG_FP32, WG_BF16 or WG_FP16");
    if (p->steps < 0 || p->steps > kMuonMaxSteps) return set_err(WG_ERR_INVALID_ARGUMENT, "steps must be 0..16");
    if (!muon_factors_ok(*p))
        return set_err(WG_ERR_INVALID_ARGUMENT, "mu must be in [0, 1), dampening in [0, 1], eps >= 0, and every factor finite");
    pl->p = *p;
    wg_muon_problem& q = pl->p;
    if (q.ld == 0) q.ld = q.cols;
    if (q.ld < q.cols) return set_err(WG_ERR_INVALID_ARGUMENT, "ld must be 0 or at least cols");
    const bool far = q.ld > kMaxSpan / q.rows;
    if (!far && (q.batch_stride == 0 || q.batch == 1)) q.batch_stride = (long long)q.rows * q.ld;
    if (far || q.batch_stride > kMaxSpan / q.batch)
        return set_err(WG_ERR_INVALID_ARGUMENT, "ld or batch_stride is larger than any memory");
    // Matrices after one another, or side by side (a matrix per head of a fused weight).
    const bool apart = q.batch_stride >= (long long)(q.rows - 1) * q.ld + q.cols;
    const bool beside = q.batch_stride >= q.cols && q.ld >= (long long)(q.batch - 1) * q.batch_stride + q.cols;
    if (q.batch > 1 && !apart && !beside)
        return set_err(WG_ERR_INVALID_ARGUMENT, "ld or batch_stride makes rows overlap");
    static const float kDefault[3] = {3.4445f, -4.7750f, 2.0315f};
    double smax = 1.0;
    for (int i = 0; i < q.steps; ++i) {
        memcpy(pl->coef[i], q.coef ? q.coef + 3 * i : kDefault, sizeof kDefault);
        const float* k = pl->coef[i];
        if (!isfinite(k[0]) || !isfinite(k[1]) || !isfinite(k[2]))
            return set_err(WG_ERR_INVALID_ARGUMENT, "coef must be finite");
        double grown, poly;
        step_range(pl->coef[i], smax, &grown, &poly);
        if (!(grown <= 4.0) || !(poly <= 48.0))
            return set_err(WG_ERR_INVALID_ARGUMENT, "coef lets a singular value grow above 4");
        smax = std::max(grown, 1e-3);
    }
    q.coef = nullptr;
    pl->m = std::min(q.rows, q.cols);
    pl->ldx = (q.cols + 7) / 8 * 8;
    pl->ldm = (pl->m + 7) / 8 * 8;
    const long long n = (long long)q.rows * q.cols;
    // Eight CTAs of the elementwise kernels per SM, of 2048 elements at least.
    pl->nparts = (int)std::max(1LL, std::min<long long>(std::max(1, kMuonMaxParts / q.batch), (n + 2047) / 2048));
    size_t o = 0;
    pl->gram = q.steps > 0 && pl->m <= 128;
    if (pl->gram) {
        muon_gram_plan(pl);
        // X between launches; of one, nothing (callers need no case for a form without a workspace).
        pl->bytes = pl->launches > 1 ? up256((size_t)q.batch * q.rows * q.cols * 4) : 256;
        return WG_OK;
    }
    pl->two = muon_single_error(pl->coef, q.steps) > 100.0;
    const size_t x = up256((size_t)q.batch * q.rows * pl->ldx * 2), a = up256((size_t)q.batch * pl->m * pl->ldm * 2);
    pl->off_part = o, o += up256((size_t)q.batch * pl->nparts * 4);
    if (q.steps > 0) {
        pl->off_x[0] = o, o += x;
        pl->off_x[1] = o, o += x;
        pl->off_xlo[0] = pl->off_xlo[1] = o, o += x;
        pl->off_a = o, o += a;
        pl->off_b = o, o += a;
        if (pl->two) {
            pl->off_xlo[1] = o, o += x;
            pl->off_alo = o, o += a;
            pl->off_blo = o, o += a;
        }
        pl->pairs = std::max(1, num_sms() / 2);
        pl->off_sums = o, o += (size_t)pl->pairs * 2 * 256 * 256 * 4;
        pl->off_arrived = o, o += up256((size_t)pl->pairs * 2 * wg::kMgEpiWarps * 4);
    }
    pl->bytes = o;
    return WG_OK;
}

// Plans are a pure function of the sizes, types and strides, the coefficients and the SM
// count; successful ones are cached, so that repeated calls skip the range checks.  (Where
// the cache cannot have memory, the plan is made anew.)  The factors, of which a learning
// rate changes from step to step, are the call's own.
int muon_plan(const wg_muon_problem* p, MuonPlan* pl)
{
    if (!p || p->steps < 0 || p->steps > kMuonMaxSteps || !muon_factors_ok(*p)) return make_muon_plan(p, pl);
    static std::mutex mu;
    static std::map<std::string, MuonPlan> cache;
    std::string key;
    try {
        // (The record's members one by one: what lies between them may be anything.)
        const auto add = [&key](const auto& v) { key.append(reinterpret_cast<const char*>(&v), sizeof v); };
        key.reserve(384);
        add(p->batch), add(p->rows), add(p->cols), add(p->ld), add(p->batch_stride);
        add(p->grad_dtype), add(p->out_dtype), add(p->weight_dtype), add(p->steps), add(p->nesterov);
        add(num_sms());
        if (p->coef) key.append(reinterpret_cast<const char*>(p->coef), (size_t)p->steps * 3 * sizeof(float));
        std::lock_guard<std::mutex> lk(mu);
        const auto it = cache.find(key);
        if (it != cache.end()) {
            *pl = it->second;
            wg_muon_problem& q = pl->p;
            q.mu = p->mu, q.dampening = p->dampening, q.eps = p->eps;
            q.scale = p->scale, q.lr = p->lr, q.weight_decay = p->weight_decay;
            return WG_OK;
        }
    } catch (...) {
        return make_muon_plan(p, pl);
    }
    const int st = make_muon_plan(p, pl);
    if (st) return st;
    try {
        std::lock_guard<std::mutex> lk(mu);
        if (cache.size() > 1024) cache.clear();
        cache.emplace(std::move(key), *pl);
    } catch (...) {
    }
    return WG_OK;
}

template <int P, bool VEC>
int muon_gram_launch(const MuonPlan& pl, const wg::GramParams& g, cudaStream_t s)
{
    const int smem = wg::gram_smem_bytes(P);
    const int st = wg::ensure_smem(wg::muon_gram_kernel<P, VEC>, smem);
    if (st) return st;
    if (g.C > 8) {  // beyond the portable cluster size
        const cudaError_t e = cudaFuncSetAttribute(wg::muon_gram_kernel<P, VEC>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return cuda_fail("cudaFuncSetAttribute", e);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    unsigned na = 0;
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = (unsigned)g.C;
    attr[na].val.clusterDim.y = attr[na].val.clusterDim.z = 1;
    ++na;
    wg::pdl_config(&cfg, attr, &na, s);
    cfg.gridDim = dim3((unsigned)(pl.blocks * g.C));
    cfg.blockDim = dim3(wg::kGramBlock);
    cfg.dynamicSmemBytes = (size_t)smem;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, wg::muon_gram_kernel<P, VEC>, g);
    return e == cudaSuccess ? WG_OK : cuda_fail("muon_gram_kernel launch", e);
}

// fp16 matrices [batch][rows][cols], read in boxes of 64 columns by `box` rows.
int muon_map(CUtensorMap* tm, void* base, int cols, int rows, int batch, int ld, long long bs, int box)
{
    wg::EncodeTiledFn fn = wg::encode_fn();
    if (!fn) return set_err(WG_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)bs * 2};
    const cuuint32_t bx[3] = {64, (cuuint32_t)box, 1}, es[3] = {1, 1, 1};
    const CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dims, strides, bx, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_err(WG_ERR_CUDA, "cuTensorMapEncodeTiled failed with CUresult " + std::to_string((int)r));
    return WG_OK;
}

// A matrix of the workspace as an operand (lo: its second values).
struct MuonOperand {
    void *base, *lo;
    int cols, rows, ld;
    long long bs;
};

template <int BN, int KIND, bool TWO>
int muon_product_launch(const MuonPlan& pl, const wg::MuonParams& p, wg::MuonProduct& g, const MuonOperand& oa,
                        const MuonOperand& ob, cudaStream_t s)
{
    const int used = g.whole ? g.pairs : std::max(g.cut, 1);
    wg::MgMaps<TWO> maps;
    int st = WG_OK;
    for (int i = 0; !st && i < (TWO ? 4 : 2); ++i) {
        const MuonOperand& o = i & 1 ? ob : oa;
        const int box = (i & 1 ? g.b_mn : g.a_mn) ? 64 : i & 1 ? BN / 2 : 128;
        st = muon_map(&maps.m[i], i < 2 ? o.base : o.lo, o.cols, o.rows, p.batch, o.ld, o.bs, box);
    }
    if (!st) st = wg::ensure_smem(wg::muon_product_kernel<BN, KIND, TWO>, wg::Mg<BN>::kSmem);
    if (st) return st;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    unsigned na = 0;
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = 2;
    attr[na].val.clusterDim.y = attr[na].val.clusterDim.z = 1;
    ++na;
    wg::pdl_config(&cfg, attr, &na, s);
    cfg.gridDim = dim3((unsigned)(2 * used));
    cfg.blockDim = dim3(wg::kMgThreads);
    cfg.dynamicSmemBytes = wg::Mg<BN>::kSmem;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, wg::muon_product_kernel<BN, KIND, TWO>, maps, p, g);
    return e == cudaSuccess ? WG_OK : cuda_fail("muon_product_kernel launch", e);
}

template <int BN>
int muon_product_bn(const MuonPlan& pl, const wg::MuonParams& p, wg::MuonProduct& g, const MuonOperand& oa,
                    const MuonOperand& ob, cudaStream_t s)
{
    switch (g.kind) {
        case wg::kMuonA: return muon_product_launch<BN, wg::kMuonA, false>(pl, p, g, oa, ob, s);
        case wg::kMuonB: return muon_product_launch<BN, wg::kMuonB, false>(pl, p, g, oa, ob, s);
        case wg::kMuonX: return muon_product_launch<BN, wg::kMuonX, false>(pl, p, g, oa, ob, s);
        case wg::kMuonLast: return muon_product_launch<BN, wg::kMuonLast, false>(pl, p, g, oa, ob, s);
        default: return muon_product_launch<BN, wg::kMuonLastAny, false>(pl, p, g, oa, ob, s);
    }
}

// Products of two values each have one form of results.
template <int BN>
int muon_product_two(const MuonPlan& pl, const wg::MuonParams& p, wg::MuonProduct& g, const MuonOperand& oa,
                     const MuonOperand& ob, cudaStream_t s)
{
    switch (g.kind) {
        case wg::kMuonA: return muon_product_launch<BN, wg::kMuonA, true>(pl, p, g, oa, ob, s);
        case wg::kMuonB: return muon_product_launch<BN, wg::kMuonB, true>(pl, p, g, oa, ob, s);
        case wg::kMuonX: return muon_product_launch<BN, wg::kMuonX, true>(pl, p, g, oa, ob, s);
        default: return muon_product_launch<BN, wg::kMuonLastAny, true>(pl, p, g, oa, ob, s);
    }
}

// One product over a sum of length K.
int muon_product(const MuonPlan& pl, const wg::MuonParams& p, wg::MuonProduct& g, const MuonOperand& oa,
                 const MuonOperand& ob, int K, cudaStream_t s)
{
    g.kb1 = (K + 63) / 64, g.kb = pl.two ? 3 * g.kb1 : g.kb1;
    g.pairs = pl.pairs;
    // The tiles' width, whether a symmetric product takes only the tiles on and
    // below the diagonal, and the parts that the leftover tiles are cut into, by
    // the time of the longest pair in us, as measured: a 64-long block of sums takes
    // 0.33 for 256 columns (the rate of cuBLAS) and 0.22 for 128 (0.27 when all pairs
    // are busy: their operands are twice the bytes per MMA); a tile's mirror image 1;
    // parts that meet in memory 2, and 3 (256 columns) or 1.3 each (the Gram matrix of
    // 512 x 32000: 142 us whole, 52 in eight parts).  Beside whole waves of tiles the others are not cut: their parts'
    // way through memory is slow beside the tiles' operands (8 of 1024 x 1024: 349 us
    // whole, 583 in four parts).
    const int tm = (g.M + 255) / 256, sym = g.sym;
    double best = 1e30;
    int bn = 256, parts = 1;
    for (int w = 1; w <= 2; ++w)
        for (int half = 0; half <= sym; ++half) {
            const int tn = (g.N * w + 255) / 256;
            const long long per = half ? (long long)w * (tm * (tm + 1) / 2) - (w * tm - tn) : (long long)tm * tn;
            const long long tiles = p.batch * per, full = tiles / g.pairs, rest = tiles % g.pairs;
            const double unit = w == 1 ? 0.33 : full ? 0.27 : 0.22;
            for (int n = 1; n <= 16; ++n) {
                if (n > 1 && (rest == 0 || rest * n > g.pairs || g.kb < 4 * n || full)) continue;
                const double t = (full + (rest ? 1.0 / n : 0.0)) * g.kb * unit + half + (n > 1 ? 2 + (w == 1 ? 3.0 : 1.3) * n : 0);
                if (t < best) best = t, bn = 256 / w, parts = n, g.sym = half, g.per = (int)per, g.tn = tn;
            }
        }
    g.tm = tm;
    g.tiles = p.batch * g.per;
    g.whole = g.tiles / g.pairs * g.pairs;
    g.cut = std::max(1, (g.tiles - g.whole) * parts);
    // What truncation takes of the products of first values, by the parts that they are in.
    double back = 0.0;
    for (int i = 0; pl.two && i < parts; ++i) {
        const int k0 = std::max(2 * g.kb1, g.kb * i / parts), k1 = g.kb * (i + 1) / parts;
        if (k1 > k0) back += (muon_put_back(K / 16.0 * (k1 - k0) / g.kb1) - 1.0) * (k1 - k0) / g.kb1;
    }
    g.sums = (float)(0x1p-10 * (1.0 + back));
    if (pl.two) return bn == 256 ? muon_product_two<256>(pl, p, g, oa, ob, s) : muon_product_two<128>(pl, p, g, oa, ob, s);
    return bn == 256 ? muon_product_bn<256>(pl, p, g, oa, ob, s) : muon_product_bn<128>(pl, p, g, oa, ob, s);
}

// The multiple t of the identity that a step, `left` before the last, moves from a to B:
// in the last step minus B's eigenvalue for a singular value of 1, about where all are
// by then, and 0.4 of it in the step before, to quarters (exact in fp16).  The other
// steps still have small singular values, into which the roundings of t X in fp16
// would come.  X's error in a simulation of every rounding (300 x 800 to 400 x 420):
// full rank 1.5-1.9e-3 without, 1.0-1.3e-3 with; rank m / 16 and noise 0.6e-3 and
// 1.3e-3; rank one 0.3e-3 and 1.5e-3; t in all steps 1e-3, 3e-2 and 0.1.
float muon_shift(const float* c, int left)
{
    if (left > 1 || fabsf(c[2]) < 1e-3f) return 0.f;
    const float t = -(c[1] + c[2]) * (left ? 0.4f : 1.f);
    return fminf(fmaxf(floorf(4.f * t + 0.5f) * 0.25f, 0.f), 4.f);
}

int muon_run(const MuonPlan& pl, const void* grad, void* momentum, void* weight, void* out, char* ws, cudaStream_t s)
{
    const wg_muon_problem& q = pl.p;
    wg::MuonParams p = {};
    p.batch = q.batch, p.rows = q.rows, p.cols = q.cols, p.ld = p.gld = q.ld, p.bs = p.gbs = q.batch_stride;
    p.grad = grad, p.mom = static_cast<float*>(momentum), p.weight = weight, p.out = out;
    p.grad_dtype = q.grad_dtype, p.out_dtype = q.out_dtype, p.weight_dtype = q.weight_dtype;
    p.nesterov = q.nesterov, p.mu = q.mu, p.gain = 1.f - q.dampening, p.eps = q.eps;
    p.scale = q.scale, p.keep = 1.f - q.lr * q.weight_decay, p.lr = q.lr;
    p.ldx = pl.ldx, p.m = pl.m, p.ldm = pl.ldm;
    p.xs = (long long)q.rows * pl.ldx, p.ms = (long long)pl.m * pl.ldm;
    const bool al = q.cols % 8 == 0 && q.ld % 8 == 0 && q.batch_stride % 8 == 0;
    if (pl.gram) {
        for (int n = 0; n < pl.launches; ++n) {
            const bool start = n == 0, end = n == pl.launches - 1;
            wg::GramParams g = pl.g;
            g.p = p;
            g.steps = pl.first[n + 1] - pl.first[n];
            std::copy(pl.g.step + pl.first[n], pl.g.step + pl.first[n + 1], g.step);
            g.parts = momentum || q.grad_dtype == WG_FP32 ? 3 : q.grad_dtype == WG_FP16 ? 2 : 1;
            if (!start) {  // X, packed
                g.raw = 1, g.parts = 3;
                g.p.grad = ws, g.p.grad_dtype = WG_FP32, g.p.mom = nullptr;
                g.p.gld = q.cols, g.p.gbs = (long long)q.rows * q.cols;
            }
            if (!end) {  // (A CTA has read an element of X before it writes it, and no other CTA reads it.)
                g.p.out = ws, g.p.out_dtype = WG_FP32, g.p.weight = nullptr;
                g.p.scale = (float)muon_put_back(pl.m / 16.0);
                g.p.ld = q.cols, g.p.bs = (long long)q.rows * q.cols;
            }
            const bool vec = (start ? al && aligned16(grad) && aligned16(momentum) : q.cols % 8 == 0) &&
                             (end ? al && aligned16(weight) && aligned16(out) : q.cols % 8 == 0);
            const int st = pl.P == 64 ? vec ? muon_gram_launch<64, true>(pl, g, s) : muon_gram_launch<64, false>(pl, g, s)
                                      : vec ? muon_gram_launch<128, true>(pl, g, s) : muon_gram_launch<128, false>(pl, g, s);
            if (st) return st;
        }
        return WG_OK;
    }
    p.part = reinterpret_cast<float*>(ws + pl.off_part), p.nparts = pl.nparts;
    if (q.steps > 0) {
        for (int i = 0; i < 2; ++i) p.x[i] = reinterpret_cast<__half*>(ws + pl.off_x[i]);
        for (int i = 0; i < 2; ++i) p.xlo[i] = reinterpret_cast<__half*>(ws + pl.off_xlo[i]);
        p.a = reinterpret_cast<__half*>(ws + pl.off_a), p.b = reinterpret_cast<__half*>(ws + pl.off_b);
        if (pl.two) p.alo = reinterpret_cast<__half*>(ws + pl.off_alo), p.blo = reinterpret_cast<__half*>(ws + pl.off_blo);
    }
    if (q.steps > 0)
        p.arrived = reinterpret_cast<int*>(ws + pl.off_arrived), p.narrived = pl.pairs * 2 * wg::kMgEpiWarps;
    const bool ivec = al && aligned16(grad) && aligned16(momentum), ovec = al && aligned16(weight) && aligned16(out);
    const dim3 egrid(pl.nparts, q.batch);
    // Division of vector indexes (below 2^31) by the vectors of a row.
    const auto rows_of = [&](bool vec) {
        p.nv = vec ? q.cols / 8 : q.cols;
        int bits = 0;
        while ((1LL << bits) < p.nv) ++bits;
        p.nv_shift = 31 + bits;
        p.nv_mul = (unsigned)(((1ULL << p.nv_shift) + p.nv - 1) / p.nv);
    };
    const bool nvec = ivec && (q.steps > 0 || ovec);
    rows_of(ivec);
    int st = launch("muon_momentum_kernel launch", ivec ? wg::muon_momentum_kernel<8> : wg::muon_momentum_kernel<1>,
                    egrid, dim3(256), 0, s, p);
    rows_of(nvec);
    if (!st)
        st = launch("muon_normalize_kernel launch",
                    nvec ? wg::muon_normalize_kernel<8> : wg::muon_normalize_kernel<1>, egrid,
                    dim3(256), 0, s, p, (int)(q.steps == 0));
    if (st || q.steps == 0) return st;
    const bool wide = q.rows <= q.cols;
    const MuonOperand x[2] = {{p.x[0], p.xlo[0], q.cols, q.rows, pl.ldx, p.xs}, {p.x[1], p.xlo[1], q.cols, q.rows, pl.ldx, p.xs}};
    const MuonOperand ma = {p.a, p.alo, pl.m, pl.m, pl.ldm, p.ms}, mb = {p.b, p.blo, pl.m, pl.m, pl.ldm, p.ms};
    for (int i = 0; i < q.steps; ++i) {
        const int in = i & 1;
        wg::MuonProduct g = {};
        g.a = pl.coef[i][0], g.b = pl.coef[i][1], g.c = pl.coef[i][2];
        const float t = pl.two ? 0.f : muon_shift(pl.coef[i], q.steps - 1 - i);
        if (t > 0.f) g.a -= t, g.tc = t * 0x1p20f / g.c;
        g.xin = in;
        g.part = reinterpret_cast<float*>(ws + pl.off_sums), g.arrived = p.arrived;
        g.kind = wg::kMuonA, g.M = g.N = pl.m, g.sym = 1;
        g.a_mn = g.b_mn = !wide;
        if ((st = muon_product(pl, p, g, x[in], x[in], std::max(q.rows, q.cols), s))) return st;
        g.kind = wg::kMuonB, g.a_mn = g.b_mn = 0;
        if ((st = muon_product(pl, p, g, ma, ma, pl.m, s))) return st;
        g.kind = i < q.steps - 1 ? wg::kMuonX : ovec ? wg::kMuonLast : wg::kMuonLastAny, g.M = q.rows, g.N = q.cols, g.sym = 0;
        g.b_mn = wide;
        st = wide ? muon_product(pl, p, g, mb, x[in], pl.m, s) : muon_product(pl, p, g, x[in], mb, pl.m, s);
        if (st) return st;
    }
    return WG_OK;
}

// Whether [a, a + na) and [b, b + nb) share bytes (NULL: nothing there).
bool overlap(const void* a, long long na, const void* b, long long nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x && y && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// ---------------------------------------------------------------- embedding
struct EmbPlan {
    wg_embedding_problem p;
    bool small;         // the one-kernel form
    int R;              // table rows of a CTA (of the sort)
    int W, tiles;       // entries of a window, column tiles
    long long windows;  // windows of the sorted list
    size_t off_meta, off_count, off_list, off_row, off_cross, off_part, bytes;
};

int emb_plan(const wg_embedding_problem* p, EmbPlan* pl)
{
    if (!p) return set_err(WG_ERR_INVALID_ARGUMENT, "problem is NULL");
    // (Numbers of rows and columns are 32-bit, those past the end of a CTA's share too.)
    if (p->tokens < 0 || p->tokens > 0x7fffff00LL || p->vocab < 1 || p->vocab > 0x7fff0000 || p->dim < 1 ||
        p->dim > 0x7fff0000)
        return set_err(WG_ERR_INVALID_ARGUMENT, "tokens must be in 0..2^31-256, vocab and dim in 1..2^31-65536");
    if (!dtype_ok(p->table_dtype) || !dtype_ok(p->out_dtype))
        return set_err(WG_ERR_INVALID_ARGUMENT, "table_dtype and out_dtype must be WG_FP32, WG_BF16 or WG_FP16");
    if (p->token_bits != 32 && p->token_bits != 64)
        return set_err(WG_ERR_INVALID_ARGUMENT, "token_bits must be 32 or 64");
    if (p->padding_token < -1 || p->padding_token >= p->vocab)
        return set_err(WG_ERR_INVALID_ARGUMENT, "padding_token must be -1 or a row of the table");
    if (!isfinite(p->scale)) return set_err(WG_ERR_INVALID_ARGUMENT, "scale must be finite");
    pl->p = *p;
    wg_embedding_problem& q = pl->p;
    if (q.ld_table == 0) q.ld_table = q.dim;
    if (q.ld_out == 0) q.ld_out = q.dim;
    if (q.ld_table < q.dim || q.ld_out < q.dim)
        return set_err(WG_ERR_INVALID_ARGUMENT, "ld_table and ld_out must be 0 or at least dim");
    if (q.ld_table > kMaxSpan / q.vocab || q.ld_out > kMaxSpan / std::max(q.tokens, 1LL))
        return set_err(WG_ERR_INVALID_ARGUMENT, "ld_table or ld_out is larger than any memory");
    // Few tokens of a small table take one kernel: 512 tokens of 8192 x 512 in fp32 9 us
    // against 14 in three, 1000 of 8192 x 1024 in bf16 14 against 15; 100 of 16384 x 1024
    // 14 both ways, 64 of 32768 x 1024 24 against 17 (the SMs that have matches to place
    // fall behind those that write zeros).
    pl->small = q.tokens <= wg::kEmbSmallTokens && q.tokens * q.dim * esize(q.out_dtype) <= (2 << 20) &&
                (long long)q.vocab * q.dim * esize(q.table_dtype) <= (16 << 20);
    // One CTA of the sort per SM, unless its counters would not fit (two of the one-kernel form's).
    const int per_sm = pl->small ? 2 : 1;
    pl->R = std::min((q.vocab + per_sm * num_sms() - 1) / (per_sm * num_sms()),
                     pl->small ? wg::kEmbSmallMaxRows : wg::kEmbSortMaxRows);
    // Windows of 32 entries, or of 16 or 8 while those make fewer than 16 warps per SM.
    pl->tiles = (q.dim + wg::kEmbTile - 1) / wg::kEmbTile;
    for (pl->W = 32; pl->W > 8 && q.tokens / pl->W * pl->tiles < 16LL * num_sms();) pl->W /= 2;
    pl->windows = (q.tokens + pl->W - 1) / pl->W;
    if (pl->windows * pl->tiles > 0x7fffffffLL)
        return set_err(WG_ERR_NOT_SUPPORTED, "more tokens by columns than one launch covers");
    size_t o = 0;
    pl->off_meta = o, o += 256;
    pl->off_count = o, o += up256((size_t)q.vocab * 4);
    pl->off_list = o, o += up256((size_t)q.tokens * 4);
    pl->off_row = o, o += up256((size_t)q.tokens * 4);
    pl->off_cross = o, o += up256((size_t)pl->windows * 16);
    pl->off_part = o, o += up256((size_t)pl->windows * 2 * q.dim * 4);
    pl->bytes = o;
    return WG_OK;
}

wg::EmbParams emb_params(const EmbPlan& pl, const void* token, const void* in, void* out)
{
    const wg_embedding_problem& q = pl.p;
    wg::EmbParams p = {};
    p.T = q.tokens, p.V = q.vocab, p.D = q.dim, p.ld_table = q.ld_table, p.ld_out = q.ld_out;
    p.token = token, p.token64 = q.token_bits == 64, p.padding = q.padding_token, p.scale = q.scale;
    p.in = in, p.out = out;
    return p;
}

// `written`: the one of table and out that the call writes.
int emb_check(const EmbPlan& pl, const void* token, const void* table, const void* out, const void* written)
{
    const wg_embedding_problem& q = pl.p;
    if ((q.tokens > 0 && (!token || !out)) || !table)
        return set_err(WG_ERR_INVALID_ARGUMENT, "token, table and out (or dy and dtable) must be non-NULL device pointers");
    if (!aligned_to(token, q.token_bits / 8) || !aligned_to(table, esize(q.table_dtype)) ||
        !aligned_to(out, esize(q.out_dtype)))
        return set_err(WG_ERR_MISALIGNED, "a pointer is not aligned to its elements");
    if (q.tokens == 0) return WG_OK;
    const long long nt = ((q.vocab - 1) * q.ld_table + q.dim) * esize(q.table_dtype);
    const long long no = ((q.tokens - 1) * q.ld_out + q.dim) * esize(q.out_dtype);
    if (overlap(table, nt, out, no) || overlap(written, written == out ? no : nt, token, q.tokens * (q.token_bits / 8)))
        return set_err(WG_ERR_INVALID_ARGUMENT, "token, table and out (or dy and dtable) must not overlap");
    return WG_OK;
}

template <typename TT, typename TO>
int emb_lookup_t(const EmbPlan& pl, const wg::EmbParams& p, cudaStream_t s)
{
    constexpr int V = sizeof(TT) == 4 || sizeof(TO) == 4 ? 4 : 8;
    const auto fits = [&](int v) {
        return p.D % v == 0 && p.ld_table % v == 0 && p.ld_out % v == 0 && aligned_to(p.in, v * (int)sizeof(TT)) &&
               aligned_to(p.out, v * (int)sizeof(TO));
    };
    const auto blocks = [&](long long n) {
        return dim3((unsigned)std::max(1LL, std::min<long long>((n + 255) / 256, 16LL * num_sms())));
    };
    if (fits(V))
        return launch("emb_lookup_kernel launch", wg::emb_lookup_kernel<TT, TO, V>, blocks(p.T * (p.D / V)), dim3(256), 0, s, p);
    const long long n = 32 * p.T * ((p.D + wg::kEmbLookCols - 1) / wg::kEmbLookCols);
    return launch("emb_lookup_any_kernel launch",
                  fits(2) ? wg::emb_lookup_any_kernel<TT, TO, 2> : wg::emb_lookup_any_kernel<TT, TO, 1>, blocks(n), dim3(256),
                  0, s, p);
}

template <typename TG, typename TY, int V>
int emb_bwd_v(const EmbPlan& pl, const wg::EmbParams& p, cudaStream_t s)
{
    if (pl.small) {
        const int smem = (2 * pl.R + 3 * (int)p.T) * 4;
        const int st = wg::ensure_smem(wg::emb_small_kernel<TG, TY, V>, smem);
        return st ? st
                  : launch("emb_small_kernel launch", wg::emb_small_kernel<TG, TY, V>, dim3((p.V + pl.R - 1) / pl.R),
                           dim3(wg::kEmbSmallThreads), smem, s, p);
    }
    const int smem = wg::kEmbSortWarps * (pl.R + p.keep) * 4;
    int st = wg::ensure_smem(wg::emb_sort_kernel<TG>, smem);
    if (!st)
        st = launch("emb_sort_kernel launch", wg::emb_sort_kernel<TG>, dim3((p.V + pl.R - 1) / pl.R),
                    dim3(wg::kEmbSortThreads), smem, s, p);
    if (st || p.T == 0) return st;
    // A warp per item; CTAs of two warps while there are fewer items than that fill the SMs.
    const long long items = pl.windows * p.tiles;
    const int warps = items < 16LL * num_sms() ? 2 : 8;
    const int ring = warps * wg::EmbRing<TY, V>::kBytes;
    if ((st = wg::ensure_smem(wg::emb_reduce_kernel<TG, TY, V>, ring))) return st;
    st = launch("emb_reduce_kernel launch", wg::emb_reduce_kernel<TG, TY, V>, dim3((unsigned)((items + warps - 1) / warps)),
                dim3(32 * warps), ring, s, p);
    // (A run of over 2 W entries needs as many tokens.)
    if (!st && p.T > 2 * p.W)
        st = launch("emb_join_kernel launch", wg::emb_join_kernel<TG>,
                    dim3((unsigned)std::min<long long>(4 * items, 8LL * num_sms())), dim3(32 * wg::kEmbJoinWarps), 0, s, p);
    return st;
}

template <typename TG, typename TY>
int emb_bwd_t(const EmbPlan& pl, const wg::EmbParams& p, cudaStream_t s)
{
    const bool vec = p.D % 8 == 0 && p.ld_table % 8 == 0 && p.ld_out % 8 == 0 && aligned16(p.in) && aligned16(p.out);
    return vec ? emb_bwd_v<TG, TY, 8>(pl, p, s) : emb_bwd_v<TG, TY, 1>(pl, p, s);
}

// Call f with the types of two dtypes.
template <typename A, typename F>
int with_second(int d, F f)
{
    return d == WG_FP32 ? f.template operator()<A, float>()
           : d == WG_BF16 ? f.template operator()<A, __nv_bfloat16>()
                          : f.template operator()<A, __half>();
}
template <typename F>
int with_types(int d1, int d2, F f)
{
    return d1 == WG_FP32 ? with_second<float>(d2, f)
           : d1 == WG_BF16 ? with_second<__nv_bfloat16>(d2, f)
                           : with_second<__half>(d2, f);
}

struct LookupCall {
    const EmbPlan& pl;
    const wg::EmbParams& p;
    cudaStream_t s;
    template <typename TT, typename TO>
    int operator()() const { return emb_lookup_t<TT, TO>(pl, p, s); }
};
struct BwdCall {
    const EmbPlan& pl;
    const wg::EmbParams& p;
    cudaStream_t s;
    template <typename TT, typename TO>
    int operator()() const { return emb_bwd_t<TT, TO>(pl, p, s); }
};

}  // namespace

extern "C" {

int wg_muon_workspace_size(const wg_muon_problem* p, size_t* bytes)
{
    if (!bytes) return set_err(WG_ERR_INVALID_ARGUMENT, "bytes is NULL");
    MuonPlan pl;
    const int st = muon_plan(p, &pl);
    if (!st) *bytes = pl.bytes;
    return st;
}

int wg_muon_plan_string(const wg_muon_problem* p, char* buf, size_t n)
{
    if (!buf || n == 0) return set_err(WG_ERR_INVALID_ARGUMENT, "buffer is NULL or empty");
    MuonPlan pl;
    const int st = muon_plan(p, &pl);
    if (st) return st;
    if (pl.gram)
        snprintf(buf, n, "kernel=muon_gram side=%s m=%d block=%d fold=%d blocks=%d cluster=%d chunks=%d steps=%d launches=%d "
                 "smem=%d ws=%zu",
                 p->rows <= p->cols ? "left" : "right", pl.m, pl.P, pl.g.F, pl.blocks, pl.g.C, pl.g.chunks, p->steps,
                 pl.launches, wg::gram_smem_bytes(pl.P), pl.bytes);
    else
        snprintf(buf, n, "kernel=muon_product side=%s m=%d steps=%d values=%d smem=%d ws=%zu",
                 p->rows <= p->cols ? "left" : "right", pl.m, p->steps, pl.two ? 2 : 1, wg::Mg<256>::kSmem, pl.bytes);
    return WG_OK;
}

int wg_muon_update(const wg_muon_problem* p, const void* grad, void* momentum, void* weight, void* out,
                   void* workspace, size_t ws_bytes, void* stream)
{
    MuonPlan pl;
    int st = muon_plan(p, &pl);
    if (st) return st;
    if (!grad || (!weight && !out))
        return set_err(WG_ERR_INVALID_ARGUMENT, "grad, and one of weight and out, must be non-NULL device pointers");
    if (!aligned_to(grad, esize(p->grad_dtype)) || !aligned_to(momentum, 4) ||
        !aligned_to(weight, esize(p->weight_dtype)) || !aligned_to(out, esize(p->out_dtype)))
        return set_err(WG_ERR_MISALIGNED, "a pointer is not aligned to its elements");
    const void* buf[4] = {grad, momentum, weight, out};
    const int es[4] = {esize(p->grad_dtype), 4, esize(p->weight_dtype), esize(p->out_dtype)};
    const long long span = (long long)(pl.p.batch - 1) * pl.p.batch_stride + (long long)(pl.p.rows - 1) * pl.p.ld + pl.p.cols;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(buf[i], span * es[i], buf[j], span * es[j]))
                return set_err(WG_ERR_INVALID_ARGUMENT, "grad, momentum, weight and out must not overlap");
    if ((st = check_workspace(pl.bytes, workspace, ws_bytes))) return st;
    return muon_run(pl, grad, momentum, weight, out, static_cast<char*>(workspace), static_cast<cudaStream_t>(stream));
}

int wg_embedding_lookup(const wg_embedding_problem* p, const void* token, const void* table, void* out, void* stream)
{
    EmbPlan pl;
    int st = emb_plan(p, &pl);
    if (st) return st;
    if ((st = emb_check(pl, token, table, out, out))) return st;
    if (pl.p.tokens == 0) return WG_OK;
    const wg::EmbParams e = emb_params(pl, token, table, out);
    return with_types(pl.p.table_dtype, pl.p.out_dtype, LookupCall{pl, e, static_cast<cudaStream_t>(stream)});
}

int wg_embedding_workspace_size(const wg_embedding_problem* p, size_t* bytes)
{
    if (!bytes) return set_err(WG_ERR_INVALID_ARGUMENT, "bytes is NULL");
    EmbPlan pl;
    const int st = emb_plan(p, &pl);
    if (!st) *bytes = pl.bytes;
    return st;
}

int wg_embedding_bwd_weight(const wg_embedding_problem* p, const void* token, const void* dy, void* dtable,
                            int accumulate, void* workspace, size_t ws_bytes, void* stream)
{
    EmbPlan pl;
    int st = emb_plan(p, &pl);
    if (st) return st;
    if ((st = emb_check(pl, token, dtable, dy, dtable))) return st;
    if ((st = check_workspace(pl.bytes, workspace, ws_bytes))) return st;
    wg::EmbParams e = emb_params(pl, token, dy, dtable);
    char* ws = static_cast<char*>(workspace);
    e.accumulate = accumulate != 0;
    // What shared memory is left keeps matches, of a quarter of a warp's positions at most.
    const long long per = (pl.p.tokens + 1023) / 1024 * 32;
    e.keep = (int)std::max(32LL, std::min<long long>((wg::kEmbSortMaxSmem / 4 / wg::kEmbSortWarps) - pl.R, per / 4 + 64));
    e.R = pl.R, e.W = pl.W, e.tiles = pl.tiles;
    e.meta = reinterpret_cast<int*>(ws + pl.off_meta), e.count = reinterpret_cast<int*>(ws + pl.off_count);
    e.list = reinterpret_cast<int*>(ws + pl.off_list), e.row = reinterpret_cast<int*>(ws + pl.off_row);
    e.cross = reinterpret_cast<int4*>(ws + pl.off_cross), e.part = reinterpret_cast<float*>(ws + pl.off_part);
    return with_types(pl.p.table_dtype, pl.p.out_dtype, BwdCall{pl, e, static_cast<cudaStream_t>(stream)});
}

}  // extern "C"
