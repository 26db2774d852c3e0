// C ABI entry points of the AdamW step over many tensors, of the 8-bit
// moments and of gradient clipping: validation, launch tables, launches.
#include <algorithm>
#include <cmath>
#include <exception>
#include <string>
#include <vector>

#include "../../include/mo.h"
#include "adamw.cuh"
#include "ns_plan.h"
#include "profile.h"
#include "runtime.h"

namespace mo {

int ctx_device(const mo_ctx* ctx);
char* ctx_workspace(const mo_ctx* ctx, size_t* bytes);   // null when detached
Profiler* ctx_profiler(mo_ctx* ctx);                     // null when profiling is off
mo_status ctx_fail(mo_ctx* ctx, mo_status st, const std::string& msg);

namespace {

constexpr int64_t MAX_NUMEL = (int64_t)1 << 38;   // blocks count in 31 bits

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t width(int type) { return type == AW_F32 ? 4 : 2; }
bool type_ok(int t) { return t == MO_F32 || t == MO_BF16 || t == MO_F16; }

// A refused argument: the message for mo_last_error.
struct Refused {
  std::string msg;
  mo_status status;
};

[[noreturn]] void refuse(const std::string& msg, mo_status status = MO_ERR_INVALID_ARG) { throw Refused{msg, status}; }
std::string at(int i) { return " (index " + std::to_string(i) + ")"; }

// Device memory that a call reads or writes; a call in which written memory
// is also read or written through another pointer is refused.
struct Range {
  uintptr_t lo, hi;
  bool written;
};

void add(std::vector<Range>& r, const void* p, size_t bytes, bool written) {
  if (p == nullptr || bytes == 0) return;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  r.push_back({lo, lo + bytes, written});
}

void check_apart(std::vector<Range>& r) {
  const auto less = [](const Range& a, const Range& b) { return a.lo < b.lo; };
  if (!std::is_sorted(r.begin(), r.end(), less)) std::sort(r.begin(), r.end(), less);
  uintptr_t end_any = 0, end_written = 0;
  for (const Range& x : r) {
    if (x.lo < (x.written ? end_any : end_written)) refuse("buffers overlap");
    end_any = std::max(end_any, x.hi);
    if (x.written) end_written = std::max(end_written, x.hi);
  }
}

// Checks one buffer of numel elements and notes its range.
void buffer(std::vector<Range>& r, const void* p, int64_t numel, size_t bytes, bool written, const char* name, int i) {
  if (p == nullptr) refuse(std::string("null ") + name + at(i));
  if (!aligned(p, bytes)) refuse(std::string(name) + " must be aligned to its elements" + at(i));
  add(r, p, (size_t)numel * bytes, written);
}

bool numel_ok(int64_t numel, int i) {
  if (numel < 0 || numel > MAX_NUMEL) refuse("bad numel" + at(i));
  return numel > 0;
}

size_t blocks_of(int64_t numel) { return (size_t)((numel + AW_BLOCK - 1) / AW_BLOCK); }

// Splits the list into launches of one set of types, of aligned tensors or of
// others, and of at most AW_MAX tensors.
class Tables {
 public:
  explicit Tables(bool by_output = false) : by_output_(by_output) { std::fill_n(&open_[0][0][0], 2 * 4 * 4, -1); }
  void add(const AwTensor& t) {
    // clip_grads leaves wt alone and launches by the output's type instead
    int& open = open_[t.vec][by_output_ ? t.ct : t.wt][t.gt];
    const long long blocks = (long long)blocks_of(t.numel);
    if (open < 0 || tabs_[open].n == AW_MAX || blocks_[open] + blocks > MAX_BLOCKS) {
      open = (int)tabs_.size();
      tabs_.emplace_back();
      tabs_.back().n = 0;
      blocks_.push_back(0);
    }
    tabs_[open].t[tabs_[open].n++] = t;
    blocks_[open] += blocks;
  }
  // Divides the tensors into runs, once all are in.
  void finish() {
    for (size_t k = 0; k < tabs_.size(); ++k) {
      AwTable& tab = tabs_[k];
      tab.run = run_of(blocks_[k]);
      tab.first[0] = 0;
      for (int i = 0; i < tab.n; ++i)
        tab.first[i + 1] = tab.first[i] + (unsigned)((blocks_of(tab.t[i].numel) + tab.run - 1) / tab.run);
      tab.runs = tab.first[tab.n];
    }
  }
  const std::vector<AwTable>& all() const { return tabs_; }

 private:
  static constexpr long long MAX_BLOCKS = 0x7fffffffll;
  std::vector<AwTable> tabs_;
  std::vector<long long> blocks_;
  int open_[2][4][4];              // the table that takes the next such tensor
  bool by_output_;
};

bool finite_nonneg(double x) { return std::isfinite(x) && x >= 0.0; }

AwHyper hyper(const mo_adamw_cfg& c, int64_t step) {
  if (!finite_nonneg(c.lr) || !finite_nonneg(c.eps)) refuse("lr and eps must be finite and >= 0");
  if (!(c.beta1 >= 0.0 && c.beta1 < 1.0) || !(c.beta2 >= 0.0 && c.beta2 < 1.0)) refuse("betas must be in [0, 1)");
  if (c.step_dev == nullptr && step < 1) refuse("step must be >= 1");
  if (!aligned(c.lr_dev, 4) || !aligned(c.step_dev, 8) || !aligned(c.grad_scale, 4) || !aligned(c.skip, 4))
    refuse("device scalars must be aligned to their type");
  AwHyper h = {};
  h.b1 = (float)c.beta1;
  h.c1 = (float)(1.0 - c.beta1);
  h.b2 = (float)c.beta2;
  h.c2 = (float)(1.0 - c.beta2);
  h.eps = (float)c.eps;
  h.lr = (float)c.lr;
  h.log_b1 = (float)std::log(c.beta1);
  h.log_b2 = (float)std::log(c.beta2);
  h.bias = c.bias_correction != 0;
  h.rate = (float)c.lr;
  h.root = 1.f;
  if (h.bias && c.step_dev == nullptr) {
    h.rate = (float)(c.lr / -std::expm1((double)step * std::log(c.beta1)));
    h.root = (float)(1.0 / std::sqrt(-std::expm1((double)step * std::log(c.beta2))));
  }
  h.stochastic = c.stochastic != 0;
  h.seed = c.seed;
  h.step = step;
  h.lr_dev = c.lr_dev;
  h.step_dev = reinterpret_cast<const long long*>(c.step_dev);
  h.gscale = c.grad_scale;
  h.skip = c.skip;
  return h;
}

// The fields that both forms of the step share.
template <typename T>
AwTensor step_tensor(const T& a, int i, std::vector<Range>& r) {
  if (!type_ok(a.g_type)) refuse("bad g_type" + at(i));
  if (a.w_type != MO_F32 && a.w_type != MO_BF16) refuse("w_type must be MO_F32 or MO_BF16" + at(i));
  if (!finite_nonneg(a.lr_scale) || !finite_nonneg(a.weight_decay))
    refuse("lr_scale and weight_decay must be finite and >= 0" + at(i));
  AwTensor t = {};
  t.wt = (AwType)a.w_type;
  t.gt = (AwType)a.g_type;
  t.ct = AW_NONE;
  buffer(r, a.W, a.numel, width(t.wt), true, "W", i);
  buffer(r, a.G, a.numel, width(t.gt), false, "G", i);
  if (a.copy != nullptr) {
    if (a.w_type != MO_F32 || (a.copy_type != MO_BF16 && a.copy_type != MO_F16))
      refuse("a copy is bf16 or fp16 and needs fp32 W" + at(i));
    t.ct = (AwType)a.copy_type;
    buffer(r, a.copy, a.numel, 2, true, "copy", i);
  }
  t.W = a.W;
  t.G = a.G;
  t.C = a.copy;
  t.numel = a.numel;
  t.lr_scale = a.lr_scale;
  t.wd = a.weight_decay;
  t.index = (unsigned)i;
  t.vec = aligned(a.W, 8 * width(t.wt)) && aligned(a.G, 8 * width(t.gt)) && aligned(a.copy, 16);
  return t;
}

template <typename T>
void codes(const T& a, int i, std::vector<Range>& r, bool written, AwTensor& t) {
  buffer(r, a.M8, a.numel, 1, written, "M8", i);
  buffer(r, a.V8, a.numel, 1, written, "V8", i);
  buffer(r, a.MS, (int64_t)blocks_of(a.numel), 1, written, "MS", i);
  buffer(r, a.VS, (int64_t)blocks_of(a.numel), 1, written, "VS", i);
  t.M = a.M8;
  t.V = a.V8;
  t.MS = a.MS;
  t.VS = a.VS;
  t.numel = a.numel;
  t.index = (unsigned)i;
  t.vec = t.vec && aligned(a.M8, 8) && aligned(a.V8, 8);
}

// Runs the body of an entry point: nothing is thrown across the C boundary.
// The body validates first, then calls launch() with what it launches, which
// runs with the context's device current.
template <typename F>
mo_status guarded(mo_ctx* ctx, const char* who, F body) {
  try {
    const auto launch = [ctx](auto launches) {
      DeviceScope scope;
      const cudaError_t e = scope.enter(ctx_device(ctx));
      return e == cudaSuccess ? launches() : e;
    };
    const cudaError_t e = body(launch);
    if (e != cudaSuccess) return ctx_fail(ctx, MO_ERR_CUDA, std::string(who) + ": " + cudaGetErrorString(e));
    return MO_OK;
  } catch (const Refused& r) {
    return ctx_fail(ctx, r.status, std::string(who) + ": " + r.msg);
  } catch (const std::exception& x) {
    return ctx_fail(ctx, MO_ERR_UNSUPPORTED, std::string(who) + ": " + x.what());
  }
}

mo_status check_list(mo_ctx* ctx, const char* who, const void* list, int n, const void* cfg) {
  if (ctx == nullptr) return MO_ERR_INVALID_ARG;
  if (n < 0) return ctx_fail(ctx, MO_ERR_INVALID_ARG, std::string(who) + ": n < 0");
  if (n > 0 && (list == nullptr || cfg == nullptr))
    return ctx_fail(ctx, MO_ERR_INVALID_ARG, std::string(who) + ": null list or cfg");
  return MO_OK;
}

struct ProfBind {
  explicit ProfBind(mo_ctx* c) { g_prof = c ? ctx_profiler(c) : nullptr; }
  ~ProfBind() { g_prof = nullptr; }
};

}  // namespace

}  // namespace mo

using namespace mo;

extern "C" {

mo_status adamw_step(mo_ctx* ctx, const mo_adamw_tensor* list, int n, const mo_adamw_cfg* cfg, int64_t step,
                     void* stream) {
  const char* who = "adamw_step";
  mo_status st = check_list(ctx, who, list, n, cfg);
  if (st != MO_OK || n == 0) return st;
  ProfBind prof(ctx);
  NvtxRange nvtx("mo adamw_step");
  return guarded(ctx, who, [&](auto launch) {
    const AwHyper h = hyper(*cfg, step);
    std::vector<Range> r;
    r.reserve((size_t)n * 5);
    Tables tabs;
    for (int i = 0; i < n; ++i) {
      const mo_adamw_tensor& a = list[i];
      if (!numel_ok(a.numel, i) || a.G == nullptr) continue;
      AwTensor t = step_tensor(a, i, r);
      buffer(r, a.M, a.numel, 4, true, "M", i);
      buffer(r, a.V, a.numel, 4, true, "V", i);
      t.M = a.M;
      t.V = a.V;
      t.vec = t.vec && aligned(a.M, 32) && aligned(a.V, 32);
      tabs.add(t);
    }
    check_apart(r);
    tabs.finish();
    return launch([&]() {
      cudaError_t e = cudaSuccess;
      for (const AwTable& tab : tabs.all())
        if (e == cudaSuccess) e = launch_adamw(tab, h, static_cast<cudaStream_t>(stream));
      return e;
    });
  });
}

mo_status adamw8_step(mo_ctx* ctx, const mo_adamw8_tensor* list, int n, const mo_adamw_cfg* cfg, int64_t step,
                      void* stream) {
  const char* who = "adamw8_step";
  mo_status st = check_list(ctx, who, list, n, cfg);
  if (st != MO_OK || n == 0) return st;
  ProfBind prof(ctx);
  NvtxRange nvtx("mo adamw8_step");
  return guarded(ctx, who, [&](auto launch) {
    const AwHyper h = hyper(*cfg, step);
    std::vector<Range> r;
    r.reserve((size_t)n * 7);
    Tables tabs;
    for (int i = 0; i < n; ++i) {
      const mo_adamw8_tensor& a = list[i];
      if (!numel_ok(a.numel, i) || a.G == nullptr) continue;
      AwTensor t = step_tensor(a, i, r);
      codes(a, i, r, true, t);
      tabs.add(t);
    }
    check_apart(r);
    tabs.finish();
    return launch([&]() {
      cudaError_t e = cudaSuccess;
      for (const AwTable& tab : tabs.all())
        if (e == cudaSuccess) e = launch_adamw8(tab, h, static_cast<cudaStream_t>(stream));
      return e;
    });
  });
}

mo_status adamw8_pack(mo_ctx* ctx, const mo_adamw8_moments* list, int n, const mo_pack_cfg* cfg, void* stream) {
  const char* who = "adamw8_pack";
  mo_status st = check_list(ctx, who, list, n, cfg);
  if (st != MO_OK || n == 0) return st;
  ProfBind prof(ctx);
  NvtxRange nvtx("mo adamw8_pack");
  return guarded(ctx, who, [&](auto launch) {
    AwHyper h = {};
    if (!aligned(cfg->step_dev, 8)) refuse("device scalars must be aligned to their type");
    h.stochastic = cfg->stochastic != 0;
    h.seed = cfg->seed;
    h.step = cfg->step;
    h.step_dev = reinterpret_cast<const long long*>(cfg->step_dev);
    std::vector<Range> r;
    r.reserve((size_t)n * 6);
    Tables tabs;
    for (int i = 0; i < n; ++i) {
      const mo_adamw8_moments& a = list[i];
      if (!numel_ok(a.numel, i)) continue;
      if (a.type != MO_F32 && a.type != MO_BF16) refuse("type must be MO_F32 or MO_BF16" + at(i));
      AwTensor t = {};
      t.gt = (AwType)a.type;
      buffer(r, a.M, a.numel, width(a.type), false, "M", i);
      buffer(r, a.V, a.numel, width(a.type), false, "V", i);
      t.G = a.M;
      t.C = a.V;
      t.vec = aligned(a.M, 8 * width(a.type)) && aligned(a.V, 8 * width(a.type));
      codes(a, i, r, true, t);
      tabs.add(t);
    }
    check_apart(r);
    tabs.finish();
    return launch([&]() {
      cudaError_t e = cudaSuccess;
      for (const AwTable& tab : tabs.all())
        if (e == cudaSuccess) e = launch_pack(tab, h, static_cast<cudaStream_t>(stream));
      return e;
    });
  });
}

mo_status adamw8_unpack(mo_ctx* ctx, const mo_adamw8_moments* list, int n, void* stream) {
  const char* who = "adamw8_unpack";
  mo_status st = check_list(ctx, who, list, n, list);
  if (st != MO_OK || n == 0) return st;
  ProfBind prof(ctx);
  NvtxRange nvtx("mo adamw8_unpack");
  return guarded(ctx, who, [&](auto launch) {
    std::vector<Range> r;
    r.reserve((size_t)n * 6);
    Tables tabs;
    for (int i = 0; i < n; ++i) {
      const mo_adamw8_moments& a = list[i];
      if (!numel_ok(a.numel, i)) continue;
      if (a.type != MO_F32 && a.type != MO_BF16) refuse("type must be MO_F32 or MO_BF16" + at(i));
      AwTensor t = {};
      t.wt = (AwType)a.type;
      buffer(r, a.M, a.numel, width(a.type), true, "M", i);
      buffer(r, a.V, a.numel, width(a.type), true, "V", i);
      t.W = a.M;
      t.C = a.V;
      t.vec = aligned(a.M, 8 * width(a.type)) && aligned(a.V, 8 * width(a.type));
      codes(a, i, r, false, t);
      tabs.add(t);
    }
    check_apart(r);
    tabs.finish();
    return launch([&]() {
      cudaError_t e = cudaSuccess;
      for (const AwTable& tab : tabs.all())
        if (e == cudaSuccess) e = launch_unpack(tab, static_cast<cudaStream_t>(stream));
      return e;
    });
  });
}

mo_status clip_grads(mo_ctx* ctx, const mo_grad* list, int n, const mo_clip_cfg* cfg, void* stream) {
  const char* who = "clip_grads";
  if (ctx == nullptr) return MO_ERR_INVALID_ARG;
  if (cfg == nullptr) return ctx_fail(ctx, MO_ERR_INVALID_ARG, "clip_grads: null cfg");
  mo_status st = check_list(ctx, who, list, n, cfg);
  if (st != MO_OK) return st;
  ProfBind prof(ctx);
  NvtxRange nvtx("mo clip_grads");
  return guarded(ctx, who, [&](auto launch) {
    if (!(cfg->max_norm >= 0.f)) refuse("max_norm must be >= 0");
    if (cfg->norm == nullptr || cfg->factor == nullptr) refuse("null norm or factor");
    if (!aligned(cfg->scale, 4) || !aligned(cfg->norm, 4) || !aligned(cfg->factor, 4) || !aligned(cfg->nonfinite, 4))
      refuse("device scalars must be aligned to their type");
    std::vector<Range> r;
    r.reserve((size_t)n * 2 + 3);
    add(r, cfg->norm, 4, true);
    add(r, cfg->factor, 4, true);
    add(r, cfg->nonfinite, 4, true);
    add(r, cfg->scale, 4, false);
    Tables tabs(true);
    for (int i = 0; i < n; ++i) {
      const mo_grad& a = list[i];
      if (!numel_ok(a.numel, i) || a.G == nullptr) continue;
      if (!type_ok(a.g_type) || (a.out != nullptr && !type_ok(a.out_type))) refuse("bad g_type or out_type" + at(i));
      AwTensor t = {};
      const bool in_place = cfg->apply && (a.out == nullptr || a.out == a.G);
      if (in_place && a.out != nullptr && a.out_type != a.g_type) refuse("out in place must keep G's type" + at(i));
      t.gt = (AwType)a.g_type;
      buffer(r, a.G, a.numel, width(t.gt), in_place, "G", i);
      t.G = a.G;
      t.C = const_cast<void*>(a.G);
      t.ct = t.gt;
      t.vec = aligned(a.G, 8 * width(t.gt));
      if (cfg->apply && !in_place) {
        t.ct = (AwType)a.out_type;
        buffer(r, a.out, a.numel, width(t.ct), true, "out", i);
        t.C = a.out;
        t.vec = t.vec && aligned(a.out, 8 * width(t.ct));
      }
      t.numel = a.numel;
      t.index = (unsigned)i;
      tabs.add(t);
    }
    check_apart(r);
    tabs.finish();
    size_t ws_bytes = 0;
    char* ws = ctx_workspace(ctx, &ws_bytes);
    if (ws == nullptr || ws_bytes < MO_CLIP_WORKSPACE_BYTES)
      refuse("needs an attached workspace of MO_CLIP_WORKSPACE_BYTES", MO_ERR_NO_WORKSPACE);
    ClipArgs a = {};
    a.partial = reinterpret_cast<double*>(ws + WS_HEADER);
    a.max_norm = cfg->max_norm;
    a.scale = cfg->scale;
    a.norm = cfg->norm;
    a.factor = cfg->factor;
    a.nonfinite = cfg->nonfinite;
    // several tables share the fixed number of partial sums
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int each = tabs.all().empty() ? 0 : CLIP_MAX_CTAS / (int)tabs.all().size();
    if (!tabs.all().empty() && each == 0) refuse("too many tensors");
    return launch([&]() {
      cudaError_t e = cudaSuccess;
      for (const AwTable& tab : tabs.all()) {
        if (e != cudaSuccess) break;
        const int ctas = clip_norm_ctas(tab, each);
        e = launch_clip_norm(tab, a.partial + a.parts, ctas, s);
        a.parts += ctas;
      }
      if (e == cudaSuccess) e = launch_clip_finish(a, s);
      if (cfg->apply)
        for (const AwTable& tab : tabs.all())
          if (e == cudaSuccess) e = launch_clip_scale(tab, cfg->factor, s);
      return e;
    });
  });
}

}  // extern "C"
