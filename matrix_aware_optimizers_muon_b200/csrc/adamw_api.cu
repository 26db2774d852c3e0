// C ABI entry points of the AdamW step over many tensors, of the 8-bit
// moments and of gradient clipping: validation, launch tables, launches.
#include <algorithm>
#include <cmath>
#include <exception>
#include <memory>
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

// The tables of a list: launches of one set of types, of aligned tensors or of
// others, and of at most AW_MAX tensors each.
class Tables {
 public:
  // most_run: the longest run; by_output: clip_grads leaves wt alone and
  // launches by the output's type instead
  explicit Tables(int most_run, int warps = STEP_RUNS, bool by_output = false)
      : most_run_(most_run), warps_(warps), by_output_(by_output) {
    std::fill_n(&open_[0][0][0], 2 * 4 * 4, -1);
  }
  void add(const AwTensor& t) {
    int& open = open_[t.vec == 2][by_output_ ? t.ct : t.wt][t.gt];
    const long long blocks = (long long)blocks_of(t.numel);
    if (open < 0 || tabs_[open]->n == AW_MAX || blocks_[open] + blocks > MAX_BLOCKS) {
      open = (int)tabs_.size();
      tabs_.emplace_back(new AwTable);
      tabs_.back()->n = 0;
      blocks_.push_back(0);
    }
    tabs_[open]->t[tabs_[open]->n++] = t;
    blocks_[open] += blocks;
  }
  // Divides the tensors into runs for a GPU of so many SMs, once all are in.
  void finish(int sms) {
    for (size_t k = 0; k < tabs_.size(); ++k) {
      AwTable& tab = *tabs_[k];
      tab.run = run_of(blocks_[k], most_run_, warps_, sms);
      tab.runs = 0;
      for (int i = 0; i < tab.n; ++i) {
        tab.t[i].first = tab.runs;
        tab.runs += (unsigned)((blocks_of(tab.t[i].numel) + tab.run - 1) / tab.run);
      }
    }
  }
  size_t size() const { return tabs_.size(); }
  const AwTable& operator[](size_t k) const { return *tabs_[k]; }

 private:
  static constexpr long long MAX_BLOCKS = 0x7fffffffll;
  int most_run_, warps_;
  bool by_output_;
  std::vector<std::unique_ptr<AwTable>> tabs_;
  std::vector<long long> blocks_;
  int open_[2][4][4];              // the table that takes the next such tensor
};

// Whether the first of two 8-bit moments takes noise (see mo_adamw_cfg).
bool first_by_noise(int stochastic) { return stochastic != 0 && stochastic != 2; }

bool finite_nonneg(double x) { return std::isfinite(x) && x >= 0.0; }

AwHyper hyper(const mo_adamw_cfg& c, int64_t step) {
  if (!finite_nonneg((float)c.lr) || !finite_nonneg((float)c.eps)) refuse("lr and eps must be finite (fp32) and >= 0");
  if (!(c.beta1 >= 0.0 && c.beta1 < 1.0) || !(c.beta2 >= 0.0 && c.beta2 < 1.0)) refuse("betas must be in [0, 1)");
  if (c.step_dev == nullptr && step < 1) refuse("step must be >= 1");
  if (!aligned(c.lr_dev, 4) || !aligned(c.step_dev, 8) || !aligned(c.grad_scale, 4) || !aligned(c.skip, 4))
    refuse("device scalars must be aligned to their type");
  AwHyper h = {};
  h.b1 = (float)c.beta1;
  h.c1 = (float)(1.0 - c.beta1);
  h.b2 = (float)c.beta2;
  h.c2 = (float)(1.0 - c.beta2);
  h.least_scale = 32;                                  // 2^-95 times 2^-31 or more
  for (float b : {h.b1, h.b2})
    if (b > 0.f && b < 0x1p-31f) h.least_scale = 256;
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
  h.first = first_by_noise(c.stochastic);
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
  t.vec = aligned(a.W, 8 * width(t.wt)) && aligned(a.G, 8 * width(t.gt)) && aligned(a.copy, 16) ? 2 : 1;
  return t;
}

template <typename T>
void codes(const T& a, int i, std::vector<Range>& r, AwTensor& t) {
  buffer(r, a.M8, a.numel, 1, true, "M8", i);
  buffer(r, a.V8, a.numel, 1, true, "V8", i);
  buffer(r, a.MS, (int64_t)blocks_of(a.numel), 1, true, "MS", i);
  buffer(r, a.VS, (int64_t)blocks_of(a.numel), 1, true, "VS", i);
  t.M = a.M8;
  t.V = a.V8;
  t.MS = a.MS;
  t.VS = a.VS;
  t.numel = a.numel;
  t.index = (unsigned)i;
  if (!aligned(a.M8, 8) || !aligned(a.V8, 8)) t.vec = 0;
}

// Stores a message without throwing.
mo_status failed(mo_ctx* ctx, mo_status st, const char* who, const char* what) noexcept {
  try {
    return ctx_fail(ctx, st, std::string(who) + ": " + what);
  } catch (...) {
    return st;
  }
}

// Runs the body of an entry point: nothing is thrown across the C boundary.
template <typename F>
mo_status guarded(mo_ctx* ctx, const char* who, F body) noexcept {
  try {
    const cudaError_t e = body();
    return e == cudaSuccess ? MO_OK : failed(ctx, MO_ERR_CUDA, who, cudaGetErrorString(e));
  } catch (const Refused& r) {
    return failed(ctx, r.status, who, r.msg.c_str());
  } catch (const std::exception& x) {
    return failed(ctx, MO_ERR_UNSUPPORTED, who, x.what());
  } catch (...) {
    return failed(ctx, MO_ERR_UNSUPPORTED, who, "unknown exception");
  }
}

// launches() with the context's device current.
template <typename F>
cudaError_t on_device(mo_ctx* ctx, F launches) {
  DeviceScope scope;
  const cudaError_t e = scope.enter(ctx_device(ctx));
  return e == cudaSuccess ? launches() : e;
}

template <typename F>
cudaError_t launch_all(mo_ctx* ctx, const Tables& tabs, F launch) {
  return on_device(ctx, [&]() {
    cudaError_t e = cudaSuccess;
    for (size_t k = 0; k < tabs.size() && e == cudaSuccess; ++k) e = launch(tabs[k]);
    return e;
  });
}

struct ProfBind {
  explicit ProfBind(mo_ctx* c) { g_prof = c ? ctx_profiler(c) : nullptr; }
  ~ProfBind() { g_prof = nullptr; }
};

enum ListKind { LIST_ADAMW, LIST_ADAMW8, LIST_MOMENTS, LIST_GRADS };

}  // namespace

}  // namespace mo

// A checked list with its launch tables.
struct mo_list {
  mo::ListKind kind;
  int device;
  mo::Tables tabs;
  std::vector<mo::Range> ranges;       // sorted
};

namespace mo {

namespace {

// Whether [p, p + bytes) meets a range of the list.
bool touches(const mo_list& l, const void* p, size_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  for (const Range& x : l.ranges)
    if (p != nullptr && lo < x.hi && x.lo < lo + bytes) return true;
  return false;
}

// Whether [p, p + bytes) meets memory that the list writes.  No other range of
// the list meets that: behind the first range that begins before p there is none.
bool in_written(const mo_list& l, const void* p, size_t bytes) {
  if (p == nullptr) return false;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  auto x = std::lower_bound(l.ranges.begin(), l.ranges.end(), lo + bytes, [](const Range& a, uintptr_t b) { return a.lo < b; });
  while (x != l.ranges.begin()) {
    --x;
    if (x->written && lo < x->hi) return true;
    if (x->lo < lo) return false;
  }
  return false;
}

template <typename T, typename F>
std::unique_ptr<mo_list> build(const mo_ctx* ctx, ListKind kind, const T* list, int n, Tables tabs, F fill) {
  if (n < 0) refuse("n < 0");
  if (n > 0 && list == nullptr) refuse("null list");
  std::unique_ptr<mo_list> l(new mo_list{kind, ctx_device(ctx), std::move(tabs), {}});
  l->ranges.reserve((size_t)n * 7);
  for (int i = 0; i < n; ++i)
    if (numel_ok(list[i].numel, i)) fill(list[i], i, *l);
  check_apart(l->ranges);
  l->tabs.finish(device_sm_count(l->device));
  return l;
}

std::unique_ptr<mo_list> build_adamw(const mo_ctx* ctx, const mo_adamw_tensor* list, int n) {
  return build(ctx, LIST_ADAMW, list, n, Tables(AW_RUN32), [](const mo_adamw_tensor& a, int i, mo_list& l) {
    if (a.G == nullptr) return;
    AwTensor t = step_tensor(a, i, l.ranges);
    buffer(l.ranges, a.M, a.numel, 4, true, "M", i);
    buffer(l.ranges, a.V, a.numel, 4, true, "V", i);
    t.M = a.M;
    t.V = a.V;
    if (!aligned(a.M, 32) || !aligned(a.V, 32)) t.vec = 1;
    l.tabs.add(t);
  });
}

std::unique_ptr<mo_list> build_adamw8(const mo_ctx* ctx, const mo_adamw8_tensor* list, int n) {
  return build(ctx, LIST_ADAMW8, list, n, Tables(AW_RUN), [](const mo_adamw8_tensor& a, int i, mo_list& l) {
    if (a.G == nullptr) return;
    AwTensor t = step_tensor(a, i, l.ranges);
    codes(a, i, l.ranges, t);
    l.tabs.add(t);
  });
}

// One table serves both directions: pack reads M and V through G and C, unpack
// writes them through W and C.
std::unique_ptr<mo_list> build_moments(const mo_ctx* ctx, const mo_adamw8_moments* list, int n) {
  return build(ctx, LIST_MOMENTS, list, n, Tables(AW_RUN), [](const mo_adamw8_moments& a, int i, mo_list& l) {
    if (a.type != MO_F32 && a.type != MO_BF16) refuse("type must be MO_F32 or MO_BF16" + at(i));
    AwTensor t = {};
    t.wt = t.gt = (AwType)a.type;
    buffer(l.ranges, a.M, a.numel, width(a.type), true, "M", i);
    buffer(l.ranges, a.V, a.numel, width(a.type), true, "V", i);
    t.W = a.M;
    t.G = a.M;
    t.C = a.V;
    t.vec = aligned(a.M, 8 * width(a.type)) && aligned(a.V, 8 * width(a.type)) ? 2 : 1;
    codes(a, i, l.ranges, t);
    l.tabs.add(t);
  });
}

std::unique_ptr<mo_list> build_grads(const mo_ctx* ctx, const mo_grad* list, int n) {
  return build(ctx, LIST_GRADS, list, n, Tables(AW_RUN, GRAD_RUNS, true), [](const mo_grad& a, int i, mo_list& l) {
    if (a.G == nullptr) return;
    const bool in_place = a.out == nullptr || a.out == a.G;
    if (!type_ok(a.g_type) || (a.out != nullptr && !type_ok(a.out_type))) refuse("bad g_type or out_type" + at(i));
    if (in_place && a.out != nullptr && a.out_type != a.g_type) refuse("out in place must keep G's type" + at(i));
    AwTensor t = {};
    t.gt = (AwType)a.g_type;
    t.ct = in_place ? t.gt : (AwType)a.out_type;
    buffer(l.ranges, a.G, a.numel, width(t.gt), in_place, "G", i);
    if (!in_place) buffer(l.ranges, a.out, a.numel, width(t.ct), true, "out", i);
    t.G = a.G;
    t.C = in_place ? const_cast<void*>(a.G) : a.out;
    t.vec = aligned(a.G, 8 * width(t.gt)) && aligned(t.C, 8 * width(t.ct)) ? 2 : 1;
    t.numel = a.numel;
    t.index = (unsigned)i;
    l.tabs.add(t);
  });
}

const mo_list& of_kind(const mo_ctx* ctx, const mo_list* l, ListKind kind) {
  if (l == nullptr) refuse("null list");
  if (l->kind != kind) refuse("a list made for another call");
  if (l->device != ctx_device(ctx)) refuse("a list made for another device");
  return *l;
}

template <typename T>
const T& given(const T* cfg) {
  if (cfg == nullptr) refuse("null cfg");
  return *cfg;
}

cudaError_t run_adamw(mo_ctx* ctx, const mo_list& l, const mo_adamw_cfg& cfg, int64_t step, void* stream) {
  const AwHyper h = hyper(cfg, step);
  if (in_written(l, cfg.lr_dev, 4) || in_written(l, cfg.step_dev, 8) || in_written(l, cfg.grad_scale, 4) ||
      in_written(l, cfg.skip, 4))
    refuse("buffers overlap");
  const bool eight = l.kind == LIST_ADAMW8;
  return launch_all(ctx, l.tabs, [&](const AwTable& tab) {
    return eight ? launch_adamw8(tab, h, static_cast<cudaStream_t>(stream))
                 : launch_adamw(tab, h, static_cast<cudaStream_t>(stream));
  });
}

cudaError_t run_pack(mo_ctx* ctx, const mo_list& l, const mo_pack_cfg& cfg, void* stream) {
  AwHyper h = {};
  if (!aligned(cfg.step_dev, 8)) refuse("device scalars must be aligned to their type");
  if (in_written(l, cfg.step_dev, 8)) refuse("buffers overlap");
  h.stochastic = cfg.stochastic != 0;
  h.first = first_by_noise(cfg.stochastic);
  h.seed = cfg.seed;
  h.step = cfg.step;
  h.step_dev = reinterpret_cast<const long long*>(cfg.step_dev);
  return launch_all(ctx, l.tabs,
                    [&](const AwTable& tab) { return launch_pack(tab, h, static_cast<cudaStream_t>(stream)); });
}

cudaError_t run_unpack(mo_ctx* ctx, const mo_list& l, void* stream) {
  return launch_all(ctx, l.tabs,
                    [&](const AwTable& tab) { return launch_unpack(tab, static_cast<cudaStream_t>(stream)); });
}

cudaError_t run_clip(mo_ctx* ctx, const mo_list& l, const mo_clip_cfg& cfg, void* stream) {
  if (!(cfg.max_norm >= 0.f)) refuse("max_norm must be >= 0");
  if (cfg.norm == nullptr || cfg.factor == nullptr) refuse("null norm or factor");
  const void* scalars[] = {cfg.norm, cfg.factor, cfg.nonfinite, cfg.scale};   // the last is read
  std::vector<Range> r;
  for (int k = 0; k < 4; ++k) {
    if (!aligned(scalars[k], 4)) refuse("device scalars must be aligned to their type");
    if (touches(l, scalars[k], 4)) refuse("buffers overlap");
    add(r, scalars[k], 4, k < 3);
  }
  check_apart(r);
  size_t ws_bytes = 0;
  char* ws = ctx_workspace(ctx, &ws_bytes);
  if (ws == nullptr || ws_bytes < MO_CLIP_WORKSPACE_BYTES)
    refuse("needs an attached workspace of MO_CLIP_WORKSPACE_BYTES", MO_ERR_NO_WORKSPACE);
  ClipArgs a = {};
  a.partial = reinterpret_cast<double*>(ws + WS_HEADER);
  a.max_norm = cfg.max_norm;
  a.scale = cfg.scale;
  a.norm = cfg.norm;
  a.factor = cfg.factor;
  a.nonfinite = cfg.nonfinite;
  // several tables share the fixed number of partial sums
  const int each = l.tabs.size() == 0 ? 0 : CLIP_MAX_CTAS / (int)l.tabs.size();
  if (l.tabs.size() > 0 && each == 0) refuse("too many tensors");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return on_device(ctx, [&]() {
    cudaError_t e = cudaSuccess;
    for (size_t k = 0; k < l.tabs.size() && e == cudaSuccess; ++k) {
      const int ctas = clip_norm_ctas(l.tabs[k], each);
      e = launch_clip_norm(l.tabs[k], a.partial + a.parts, ctas, s);
      a.parts += ctas;
    }
    // with one table and few sums its scale launch finishes them
    a.finish_here = cfg.apply && l.tabs.size() == 1 && a.parts <= FEW_PARTS;
    if (!a.finish_here && e == cudaSuccess) e = launch_clip_finish(a, s);
    for (size_t k = 0; k < l.tabs.size() && e == cudaSuccess && cfg.apply; ++k) e = launch_clip_scale(l.tabs[k], a, s);
    return e;
  });
}

// Makes a list of `kind` for the caller.
template <typename F>
mo_status make_list(mo_ctx* ctx, const char* who, mo_list** out, F build_it) {
  if (ctx == nullptr) return MO_ERR_INVALID_ARG;
  return guarded(ctx, who, [&]() {
    if (out == nullptr) refuse("null out");
    *out = nullptr;
    *out = build_it().release();
    return cudaSuccess;
  });
}

// An entry point that runs: profiler, range for timeline tools, errors.
template <typename F>
mo_status entry(mo_ctx* ctx, const char* who, const char* range, F body) {
  if (ctx == nullptr) return MO_ERR_INVALID_ARG;
  ProfBind prof(ctx);
  NvtxRange nvtx(range);
  return guarded(ctx, who, body);
}

}  // namespace

}  // namespace mo

using namespace mo;

extern "C" {

mo_status mo_adamw_list(mo_ctx* ctx, const mo_adamw_tensor* list, int n, mo_list** out) {
  return make_list(ctx, "adamw_step", out, [&]() { return build_adamw(ctx, list, n); });
}
mo_status mo_adamw8_list(mo_ctx* ctx, const mo_adamw8_tensor* list, int n, mo_list** out) {
  return make_list(ctx, "adamw8_step", out, [&]() { return build_adamw8(ctx, list, n); });
}
mo_status mo_moments_list(mo_ctx* ctx, const mo_adamw8_moments* list, int n, mo_list** out) {
  return make_list(ctx, "adamw8_moments", out, [&]() { return build_moments(ctx, list, n); });
}
mo_status mo_grad_list(mo_ctx* ctx, const mo_grad* list, int n, mo_list** out) {
  return make_list(ctx, "clip_grads", out, [&]() { return build_grads(ctx, list, n); });
}
void mo_list_destroy(mo_list* list) { delete list; }

mo_status adamw_step_list(mo_ctx* ctx, const mo_list* list, const mo_adamw_cfg* cfg, int64_t step, void* stream) {
  return entry(ctx, "adamw_step", "mo adamw_step",
               [&]() { return run_adamw(ctx, of_kind(ctx, list, LIST_ADAMW), given(cfg), step, stream); });
}
mo_status adamw8_step_list(mo_ctx* ctx, const mo_list* list, const mo_adamw_cfg* cfg, int64_t step, void* stream) {
  return entry(ctx, "adamw8_step", "mo adamw8_step",
               [&]() { return run_adamw(ctx, of_kind(ctx, list, LIST_ADAMW8), given(cfg), step, stream); });
}
mo_status adamw8_pack_list(mo_ctx* ctx, const mo_list* list, const mo_pack_cfg* cfg, void* stream) {
  return entry(ctx, "adamw8_pack", "mo adamw8_pack",
               [&]() { return run_pack(ctx, of_kind(ctx, list, LIST_MOMENTS), given(cfg), stream); });
}
mo_status adamw8_unpack_list(mo_ctx* ctx, const mo_list* list, void* stream) {
  return entry(ctx, "adamw8_unpack", "mo adamw8_unpack",
               [&]() { return run_unpack(ctx, of_kind(ctx, list, LIST_MOMENTS), stream); });
}
mo_status clip_grads_list(mo_ctx* ctx, const mo_list* list, const mo_clip_cfg* cfg, void* stream) {
  return entry(ctx, "clip_grads", "mo clip_grads",
               [&]() { return run_clip(ctx, of_kind(ctx, list, LIST_GRADS), given(cfg), stream); });
}

mo_status adamw_step(mo_ctx* ctx, const mo_adamw_tensor* list, int n, const mo_adamw_cfg* cfg, int64_t step,
                     void* stream) {
  return entry(ctx, "adamw_step", "mo adamw_step", [&]() {
    if (n == 0) return cudaSuccess;
    return run_adamw(ctx, *build_adamw(ctx, list, n), given(cfg), step, stream);
  });
}
mo_status adamw8_step(mo_ctx* ctx, const mo_adamw8_tensor* list, int n, const mo_adamw_cfg* cfg, int64_t step,
                      void* stream) {
  return entry(ctx, "adamw8_step", "mo adamw8_step", [&]() {
    if (n == 0) return cudaSuccess;
    return run_adamw(ctx, *build_adamw8(ctx, list, n), given(cfg), step, stream);
  });
}
mo_status adamw8_pack(mo_ctx* ctx, const mo_adamw8_moments* list, int n, const mo_pack_cfg* cfg, void* stream) {
  return entry(ctx, "adamw8_pack", "mo adamw8_pack", [&]() {
    if (n == 0) return cudaSuccess;
    return run_pack(ctx, *build_moments(ctx, list, n), given(cfg), stream);
  });
}
mo_status adamw8_unpack(mo_ctx* ctx, const mo_adamw8_moments* list, int n, void* stream) {
  return entry(ctx, "adamw8_unpack", "mo adamw8_unpack", [&]() {
    if (n == 0) return cudaSuccess;
    return run_unpack(ctx, *build_moments(ctx, list, n), stream);
  });
}
mo_status clip_grads(mo_ctx* ctx, const mo_grad* list, int n, const mo_clip_cfg* cfg, void* stream) {
  return entry(ctx, "clip_grads", "mo clip_grads",
               [&]() { return run_clip(ctx, *build_grads(ctx, list, n), given(cfg), stream); });
}

}  // extern "C"
