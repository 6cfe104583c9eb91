// extern "C" entry points declared in include/ar.h.
#include "../../include/ar.h"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <vector>

#include "exec.h"
#include "grad.h"
#include "sched.h"

static_assert(sizeof(ar_oprec) == sizeof(ar::OpRec), "ar_oprec layout");

namespace {

thread_local std::string t_msg;
thread_local int32_t t_hip = 0;

ar_status fail(ar_status st, const std::string& m) {
  t_msg = m;
  return st;
}

// Process-wide cost model for AR_AUTO / AR_KNOB_AUTO and the choices made under it.
// Default: least-squares fit of AR_EXEC_LITERAL fp32 calls on MI355X (P = 7 and 8,
// 2^10..2^22 elements, every schedule and r), one launch per step, all ranks'
// bytes through one HBM.
constexpr ar::CostModel kDefaultModel{3.52e-6, 2.10e-13, 2.07e-13, ar::F_ALL_RANKS};
std::mutex g_model_mu;
ar::CostModel g_model = kDefaultModel;
std::map<std::string, std::pair<ar::Spec, double>> g_choices;

std::string choice_key(const ar::Spec& s) {
  std::string k = std::to_string(s.P) + "/" + std::to_string(s.n) + "/" + std::to_string(s.batch) + "/" +
                  std::to_string(s.dtype) + "/" + std::to_string(s.op) + "/" + std::to_string(s.algo) + "/" +
                  std::to_string(s.knob) + "/" + std::to_string(s.coll) + "/" + std::to_string(s.steps) + "/";
  for (int g : s.groups) k += std::to_string(g) + ",";
  return k;
}

// Replace an AR_AUTO / AR_KNOB_AUTO spec by the model's choice (cached per spec).
bool resolve(ar::Spec* s, double* seconds, std::string* err) {
  std::lock_guard<std::mutex> lk(g_model_mu);
  const std::string key = choice_key(*s);
  auto it = g_choices.find(key);
  if (it == g_choices.end()) {
    ar::Spec out;
    double t = 0;
    if (!ar::select_spec(*s, g_model, &out, &t, err)) return false;
    if (g_choices.size() > 4096) g_choices.clear();
    it = g_choices.emplace(key, std::make_pair(out, t)).first;
  }
  *s = it->second.first;
  if (seconds) *seconds = it->second.second;
  return true;
}

bool to_spec(const ar_call* c, ar::Spec* s, std::string* err) {
  if (!c) { *err = "call is NULL"; return false; }
  s->P = c->P;
  s->n = c->n;
  s->batch = c->batch == 0 ? 1 : c->batch;
  s->dtype = c->dtype;
  s->op = c->op;
  s->algo = c->algo;
  s->knob = (c->algo == AR_GENERALIZED || c->algo == AR_GENERALIZED_XOR || c->algo == AR_CHAIN) ? c->knob : 0;
  s->steps = c->steps;
  s->groups.clear();
  if (c->algo == AR_AHC) {
    if (c->ngroups < 1 || !c->groups) { *err = "AHC needs ngroups >= 1 and a groups array"; return false; }
    if (c->ngroups > AR_MAX_RANKS) { *err = "too many AHC groups"; return false; }
    s->groups.assign(c->groups, c->groups + c->ngroups);
  } else if (c->algo == AR_GENERALIZED && c->ngroups != 0) {
    if (c->ngroups < 0 || !c->groups) { *err = "ngroups > 0 needs a groups array"; return false; }
    if (c->ngroups > 8) { *err = "at most 8 group factors"; return false; }
    s->groups.assign(c->groups, c->groups + c->ngroups);
  } else if (c->algo == AR_AUTO && c->ngroups != 0) {
    if (c->ngroups < 0 || !c->groups) { *err = "ngroups > 0 needs a groups array"; return false; }
    if (c->ngroups > AR_MAX_RANKS) { *err = "too many AHC groups"; return false; }
    s->groups.assign(c->groups, c->groups + c->ngroups);
    ar::Spec probe = *s;
    probe.algo = ar::A_AHC;
    if (!ar::validate_spec(probe, err)) return false;
  }
  if (c->exec < AR_EXEC_FUSED || c->exec > AR_EXEC_DAG) { *err = "unknown exec mode"; return false; }
  if (c->collective < AR_ALLREDUCE || c->collective > AR_ALL_GATHER) { *err = "unknown collective"; return false; }
  s->coll = c->collective;
  if (s->coll == AR_ALL_GATHER) s->op = ar::O_SUM;  // copies only: the op plays no part
  if (ar::is_auto(*s)) return resolve(s, nullptr, err);
  return ar::validate_spec(*s, err);
}

ar_status check_bufs(void* const* bufs, int P) {
  if (!bufs) return fail(AR_INVALID_ARGUMENT, "bufs is NULL");
  uintptr_t v[AR_MAX_RANKS];  // P was validated: 1..AR_MAX_RANKS
  for (int p = 0; p < P; ++p) {
    if (!bufs[p]) return fail(AR_INVALID_ARGUMENT, "bufs[" + std::to_string(p) + "] is NULL");
    v[p] = reinterpret_cast<uintptr_t>(bufs[p]);
  }
  std::sort(v, v + P);
  for (int p = 1; p < P; ++p)
    if (v[p] == v[p - 1]) return fail(AR_INVALID_ARGUMENT, "two ranks share one buffer");
  return AR_OK;
}

bool is_float(int32_t dtype) { return dtype == AR_FP32 || dtype == AR_BF16; }
int64_t float_bytes(int32_t dtype) { return dtype == AR_BF16 ? 2 : 4; }
constexpr int64_t kMaxElements = int64_t(1) << 48;

ar_status check_clip(const ar_clip* c, bool scale, ar::Clip* out) {
  if (!c) return fail(AR_INVALID_ARGUMENT, "clip is NULL");
  if (c->norm != AR_NORM_L2 && c->norm != AR_NORM_MAX) return fail(AR_INVALID_ARGUMENT, "unknown norm");
  if (scale) {
    if (!(c->max_norm >= 0)) return fail(AR_INVALID_ARGUMENT, "max_norm must be >= 0");
    if (!(c->eps >= 0) || std::isinf(c->eps)) return fail(AR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  }
  if (reinterpret_cast<uintptr_t>(c->workspace) % 16) return fail(AR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
  for (const void* p : {static_cast<const void*>(c->total), static_cast<const void*>(c->each),
                        static_cast<const void*>(c->known)})
    if (reinterpret_cast<uintptr_t>(p) % 4) return fail(AR_INVALID_ARGUMENT, "total, each and known must be 4-byte aligned");
  out->norm = c->norm;
  out->max_norm = c->max_norm;
  out->eps = c->eps;
  out->total = c->total;
  out->each = c->each;
  out->known = c->known;
  out->workspace = c->workspace;
  out->workspace_bytes = c->workspace_bytes;
  out->start_event = c->start_event;
  out->stop_event = c->stop_event;
  return AR_OK;
}

// Memory that a call reads, or writes.
struct Span {
  uintptr_t lo, hi;
  bool written;
};

// Whether a written span meets another. Lists mostly come in ascending order already.
bool spans_meet(std::vector<Span>& v) {
  auto by_lo = [](const Span& a, const Span& b) { return a.lo < b.lo; };
  if (!std::is_sorted(v.begin(), v.end(), by_lo)) std::sort(v.begin(), v.end(), by_lo);
  uintptr_t end = 0, written_end = 0;  // of the spans before
  for (const Span& s : v) {
    if (s.lo < (s.written ? end : written_end)) return true;
    end = std::max(end, s.hi);
    if (s.written) written_end = std::max(written_end, s.hi);
  }
  return false;
}

ar_status check_grads(const ar_grad* g, int32_t count, bool scale, std::vector<ar::Grad>* out) {
  if (count < 0 || count > AR_MAX_GRADS)
    return fail(AR_INVALID_ARGUMENT, "count must be in [0, " + std::to_string(AR_MAX_GRADS) + "]");
  if (count && !g) return fail(AR_INVALID_ARGUMENT, "grads is NULL");
  out->reserve(size_t(count));
  std::vector<Span> spans;
  if (scale) spans.reserve(2 * size_t(count));
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) {
    const ar_grad& t = g[i];
    auto bad = [&](const char* why) { return fail(AR_INVALID_ARGUMENT, "tensor " + std::to_string(i) + ": " + why); };
    if (!is_float(t.dtype)) return bad("dtype must be AR_FP32 or AR_BF16");
    if (t.n < 0 || t.n >= kMaxElements) return bad("n must be in [0, 2^48)");
    total += t.n;
    if (total >= kMaxElements) return bad("2^48 elements or more in one call");
    if (t.n && !t.data) return bad("data is NULL");
    const uintptr_t d = reinterpret_cast<uintptr_t>(t.data);
    if (d % uintptr_t(float_bytes(t.dtype))) return bad("data is not aligned to its elements");
    ar::Grad r{t.data, const_cast<void*>(t.data), t.n, t.dtype, t.dtype};
    if (scale) {
      const bool apart = t.out && t.out != t.data;
      if (t.out) {
        if (!is_float(t.out_dtype)) return bad("out_dtype must be AR_FP32 or AR_BF16");
        if (!apart && t.out_dtype != t.dtype) return bad("clipping in place keeps the type");
        const uintptr_t o = reinterpret_cast<uintptr_t>(t.out);
        if (o % uintptr_t(float_bytes(t.out_dtype))) return bad("out is not aligned to its elements");
        r.out = t.out;
        r.out_dtype = t.out_dtype;
        if (apart && t.n) spans.push_back({o, o + uintptr_t(t.n * float_bytes(t.out_dtype)), true});
      }
      if (t.n) spans.push_back({d, d + uintptr_t(t.n * float_bytes(t.dtype)), !apart});
    }
    out->push_back(r);
  }
  if (scale && spans_meet(spans)) return fail(AR_INVALID_ARGUMENT, "a tensor that is written overlaps another");
  return AR_OK;
}

// A known norm is read by every workgroup of a call that writes: it may not lie in what the call writes.
ar_status check_known(const float* known, const std::vector<ar::Grad>& g) {
  const uintptr_t k = reinterpret_cast<uintptr_t>(known);
  for (size_t i = 0; i < g.size(); ++i) {
    const uintptr_t o = reinterpret_cast<uintptr_t>(g[i].out);
    if (g[i].n && k < o + uintptr_t(g[i].n * float_bytes(g[i].out_dtype)) && o < k + sizeof(float))
      return fail(AR_INVALID_ARGUMENT, "known lies in tensor " + std::to_string(i) + "'s result");
  }
  return AR_OK;
}

ar_status check_buckets(void* const* bufs, bool with_bufs, const int64_t* n, int32_t buckets, int32_t P, int32_t dtype,
                        int32_t op, int32_t collective, ar::Buckets* out) {
  if (P < 1 || P > AR_MAX_RANKS) return fail(AR_INVALID_ARGUMENT, "P must be in [1, " + std::to_string(AR_MAX_RANKS) + "]");
  if (buckets < 0 || int64_t(buckets) * P > AR_MAX_GRADS)
    return fail(AR_INVALID_ARGUMENT, "buckets must be >= 0, and buckets * P at most " + std::to_string(AR_MAX_GRADS));
  if (!is_float(dtype)) return fail(AR_INVALID_ARGUMENT, "dtype must be AR_FP32 or AR_BF16");
  if (op != AR_SUM && op != AR_AVG) return fail(AR_INVALID_ARGUMENT, "op must be AR_SUM or AR_AVG");
  if (collective != AR_ALLREDUCE && collective != AR_REDUCE_SCATTER)
    return fail(AR_INVALID_ARGUMENT, "collective must be AR_ALLREDUCE or AR_REDUCE_SCATTER");
  if (buckets && !n) return fail(AR_INVALID_ARGUMENT, "n is NULL");
  if (buckets && with_bufs && !bufs) return fail(AR_INVALID_ARGUMENT, "bufs is NULL");
  std::vector<Span> spans;
  if (with_bufs) spans.reserve(size_t(buckets) * size_t(P));
  int64_t total = 0;
  for (int32_t b = 0; b < buckets; ++b) {
    auto bad = [&](const std::string& why) { return fail(AR_INVALID_ARGUMENT, "bucket " + std::to_string(b) + ": " + why); };
    if (n[b] < 0 || n[b] >= kMaxElements || (total += n[b]) >= kMaxElements) return bad("n must be >= 0, and below 2^48 in all");
    for (int32_t p = 0; with_bufs && n[b] && p < P; ++p) {
      const uintptr_t v = reinterpret_cast<uintptr_t>(bufs[int64_t(b) * P + p]);
      if (!v) return bad("rank " + std::to_string(p) + "'s buffer is NULL");
      if (v % uintptr_t(float_bytes(dtype))) return bad("rank " + std::to_string(p) + "'s buffer is not aligned to its elements");
      spans.push_back({v, v + uintptr_t(n[b] * float_bytes(dtype)), true});
    }
  }
  if (spans_meet(spans)) return fail(AR_INVALID_ARGUMENT, "two buffers overlap");
  *out = ar::Buckets{bufs, n, buckets, P, dtype, op, collective};
  return AR_OK;
}

ar_status finish(const ar::RunResult& r) {
  t_hip = r.hip_error;
  if (r.status) return fail(ar_status(r.status), r.message);
  t_msg.clear();
  return AR_OK;
}

// No exception crosses the C boundary: the host tables of a call may not fit memory.
template <typename F> ar_status guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    return fail(AR_INTERNAL, e.what());
  }
}

ar_status grad_call(const ar_grad* grads, int32_t count, const ar_clip* clip, bool scale, void* stream, size_t* bytes) {
  ar::Clip c;
  std::vector<ar::Grad> g;
  ar_status st = check_clip(clip, scale, &c);
  if (st == AR_OK && c.known && !scale) st = fail(AR_INVALID_ARGUMENT, "known is for ar_grad_clip");
  if (st == AR_OK && c.known && (c.total || c.each)) st = fail(AR_INVALID_ARGUMENT, "with known, total and each must be NULL");
  if (st == AR_OK && !scale && !bytes && !c.total) st = fail(AR_INVALID_ARGUMENT, "total is NULL");
  if (st == AR_OK) st = check_grads(grads, count, scale, &g);
  if (st == AR_OK && c.known) st = check_known(c.known, g);
  if (st != AR_OK) return st;
  if (bytes) {
    *bytes = ar::grad_workspace(g.data(), int64_t(g.size()), c);
    return AR_OK;
  }
  return finish(ar::run_grad(g.data(), int64_t(g.size()), c, scale, stream));
}

}  // namespace

extern "C" {

ar_status ar_set_cost_model(const ar_cost_model* m) {
  ar::CostModel cm = kDefaultModel;
  if (m) {
    if (!(std::isfinite(m->alpha) && std::isfinite(m->beta) && std::isfinite(m->gamma)) || m->alpha < 0 ||
        m->beta < 0 || m->gamma < 0)
      return fail(AR_INVALID_ARGUMENT, "alpha, beta, gamma must be finite and >= 0");
    if (m->form != AR_COST_BUSIEST_RANK && m->form != AR_COST_ALL_RANKS)
      return fail(AR_INVALID_ARGUMENT, "unknown cost form");
    cm = ar::CostModel{m->alpha, m->beta, m->gamma, m->form};
  }
  std::lock_guard<std::mutex> lk(g_model_mu);
  g_model = cm;
  g_choices.clear();
  return AR_OK;
}

ar_status ar_set_launch_blocks(int64_t max_blocks, int64_t* previous) {
  if (!ar::set_launch_blocks(max_blocks, previous))
    return fail(AR_INVALID_ARGUMENT, "max_blocks must be in [1, " + std::to_string(ar::kMaxLaunchBlocks) + "]");
  return AR_OK;
}

ar_status ar_get_cost_model(ar_cost_model* m) {
  if (!m) return fail(AR_INVALID_ARGUMENT, "model is NULL");
  std::lock_guard<std::mutex> lk(g_model_mu);
  m->alpha = g_model.alpha;
  m->beta = g_model.beta;
  m->gamma = g_model.gamma;
  m->form = g_model.form;
  m->reserved = 0;
  return AR_OK;
}

ar_status ar_select(const ar_call* call, int32_t* algo, int32_t* knob, double* predicted_seconds) {
  std::string err;
  ar::Spec spec;
  if (!to_spec(call, &spec, &err)) return fail(AR_INVALID_ARGUMENT, err);
  double t = 0;
  if (predicted_seconds) {
    ar::CostModel cm;
    {
      std::lock_guard<std::mutex> lk(g_model_mu);
      cm = g_model;
    }
    if (!ar::select_spec(spec, cm, &spec, &t, &err)) return fail(AR_INVALID_ARGUMENT, err);
    *predicted_seconds = t;
  }
  if (algo) *algo = spec.algo;
  if (knob) *knob = spec.knob;
  return AR_OK;
}

const char* ar_status_string(ar_status st) {
  switch (st) {
    case AR_OK: return "AR_OK";
    case AR_INVALID_ARGUMENT: return "AR_INVALID_ARGUMENT";
    case AR_UNSUPPORTED: return "AR_UNSUPPORTED";
    case AR_WORKSPACE_TOO_SMALL: return "AR_WORKSPACE_TOO_SMALL";
    case AR_HIP_ERROR: return "AR_HIP_ERROR";
    case AR_INTERNAL: return "AR_INTERNAL";
  }
  return "unknown status";
}

int32_t ar_last_hip_error(void) { return t_hip; }
const char* ar_last_error_message(void) { return t_msg.c_str(); }
const char* ar_version(void) { return "allreduce-schedules-mi355x 0.1 (gfx950)"; }

ar_status ar_allreduce_ex(void* const* bufs, const ar_call* call, void* stream) {
  std::string err;
  ar::Spec spec;
  if (!to_spec(call, &spec, &err)) return fail(AR_INVALID_ARGUMENT, err);
  ar_status st = check_bufs(bufs, spec.P);
  if (st != AR_OK) return st;
  ar::RunResult r = ar::run_allreduce(bufs, spec, call->exec, call->workspace, call->workspace_bytes, stream,
                                      call->start_event, call->stop_event);
  t_hip = r.hip_error;
  if (r.status) return fail(ar_status(r.status), r.message);
  t_msg.clear();
  return AR_OK;
}

ar_status ar_allreduce(void* const* bufs, int32_t P, int64_t n, int32_t dtype, int32_t op, int32_t algo,
                       int32_t knob, void* stream) {
  if (algo == AR_AHC) return fail(AR_INVALID_ARGUMENT, "AR_AHC needs group sizes: use ar_allreduce_ex");
  ar_call c;
  std::memset(&c, 0, sizeof(c));
  c.P = P;
  c.n = n;
  c.batch = 1;
  c.dtype = dtype;
  c.op = op;
  c.algo = algo;
  c.knob = knob;
  c.exec = AR_EXEC_FUSED;
  return ar_allreduce_ex(bufs, &c, stream);
}

static_assert(AR_NOALLOC_SCRATCH_BYTES == ar::kScratchBytes, "scratch size");

ar_status ar_allreduce_noalloc(void* const* bufs, const ar_call* call, void* stream) {
  std::string err;
  ar::Spec spec;
  if (!to_spec(call, &spec, &err)) return fail(AR_INVALID_ARGUMENT, err);
  if (call->exec != AR_EXEC_LITERAL)
    return fail(AR_INVALID_ARGUMENT, "the allocation-free entry point runs the literal steps: exec must be AR_EXEC_LITERAL");
  if (call->workspace) return fail(AR_INVALID_ARGUMENT, "the allocation-free entry point takes no workspace");
  ar_status st = check_bufs(bufs, spec.P);
  if (st != AR_OK) return st;
  ar::RunResult r = ar::run_noalloc(bufs, spec, stream, call->start_event, call->stop_event);
  t_hip = r.hip_error;
  if (r.status) return fail(ar_status(r.status), r.message);
  t_msg.clear();
  return AR_OK;
}

ar_status ar_reduce_scatter(void* const* bufs, int32_t P, int64_t n, int32_t dtype, int32_t op, int32_t algo,
                            void* stream) {
  if (algo == AR_AHC) return fail(AR_INVALID_ARGUMENT, "AR_AHC has no reduce-scatter half here");
  ar_call c;
  std::memset(&c, 0, sizeof(c));
  c.P = P;
  c.n = n;
  c.batch = 1;
  c.dtype = dtype;
  c.op = op;
  c.algo = algo;
  c.exec = AR_EXEC_FUSED;
  c.collective = AR_REDUCE_SCATTER;
  return ar_allreduce_ex(bufs, &c, stream);
}

ar_status ar_all_gather(void* const* bufs, int32_t P, int64_t n, int32_t dtype, int32_t algo, void* stream) {
  if (algo == AR_AHC) return fail(AR_INVALID_ARGUMENT, "AR_AHC has no all-gather half here");
  ar_call c;
  std::memset(&c, 0, sizeof(c));
  c.P = P;
  c.n = n;
  c.batch = 1;
  c.dtype = dtype;
  c.op = AR_SUM;
  c.algo = algo;
  c.exec = AR_EXEC_FUSED;
  c.collective = AR_ALL_GATHER;
  return ar_allreduce_ex(bufs, &c, stream);
}

ar_status ar_workspace_bytes(const ar_call* call, size_t* bytes) {
  std::string err;
  ar::Spec spec;
  if (!bytes) return fail(AR_INVALID_ARGUMENT, "bytes is NULL");
  if (!to_spec(call, &spec, &err)) return fail(AR_INVALID_ARGUMENT, err);
  *bytes = 0;
  if ((call->exec == AR_EXEC_FUSED && spec.algo == AR_DIRECT && spec.coll == AR_ALLREDUCE) || spec.P <= 1 ||
      spec.n == 0)
    return AR_OK;
  ar::RunResult r = ar::workspace_bytes(spec, call->exec, bytes);
  if (r.status) return fail(ar_status(r.status), r.message);
  return AR_OK;
}

ar_status ar_kernel_of(const ar_call* call, int32_t* kernel) {
  std::string err;
  ar::Spec spec;
  if (!kernel) return fail(AR_INVALID_ARGUMENT, "kernel is NULL");
  if (!to_spec(call, &spec, &err)) return fail(AR_INVALID_ARGUMENT, err);
  int k = 0;
  ar::RunResult r = ar::kernel_of(spec, call->exec, &k);
  if (r.status) return fail(ar_status(r.status), r.message);
  *kernel = k;
  return AR_OK;
}

ar_status ar_cache_stats_get(ar_cache_stats* out) {
  if (!out) return fail(AR_INVALID_ARGUMENT, "out is NULL");
  const ar::CacheStats c = ar::cache_stats();
  out->live_plans = c.live_plans;
  out->retired_plans = c.retired_plans;
  const ar::GradCache g = ar::grad_cache();
  out->workspaces = c.workspaces + g.live;
  out->retired_workspaces = c.retired_workspaces + g.retired;
  out->plan_device_bytes = c.plan_device_bytes;
  out->workspace_device_bytes = c.workspace_device_bytes + g.bytes;
  return AR_OK;
}

ar_status ar_release_cached(void) {
  return guarded([]() -> ar_status {
    ar::RunResult r = ar::grad_cache_wait();
    if (!r.status) r = ar::release_cached();
    if (r.status) {
      t_hip = r.hip_error;
      return fail(ar_status(r.status), r.message);
    }
    ar::grad_cache_free();
    return AR_OK;
  });
}

ar_status ar_schedule_build(const ar_call* call, ar_schedule** out) {
  std::string err;
  ar::Spec spec;
  if (!out) return fail(AR_INVALID_ARGUMENT, "out is NULL");
  *out = nullptr;
  if (!to_spec(call, &spec, &err)) return fail(AR_INVALID_ARGUMENT, err);
  ar::Schedule* s = ar::build_schedule(spec, &err);
  if (!s) return fail(AR_INTERNAL, err);
  *out = reinterpret_cast<ar_schedule*>(s);
  return AR_OK;
}

ar_status ar_schedule_dag_export(const ar_schedule* sh, int32_t* shared, int32_t* offsets, size_t range_cap,
                                 uint8_t* maps, size_t map_cap, int32_t* words, size_t word_cap, size_t* nranges,
                                 size_t* nmaps, size_t* nwords) {
  if (!sh) return fail(AR_INVALID_ARGUMENT, "NULL schedule");
  const ar::Schedule& s = *reinterpret_cast<const ar::Schedule*>(sh);
  if (!s.fused_ok) return fail(AR_UNSUPPORTED, "no fused program: " + s.fused_error);
  ar::DagPlan d;
  std::string err;
  if (!ar::dag_plan(s, &d, &err)) return fail(AR_UNSUPPORTED, err);
  if (shared) *shared = d.shared ? 1 : 0;
  if (nranges) *nranges = d.offsets.size();
  if (nmaps) *nmaps = d.maps.size();
  if (nwords) *nwords = d.words.size();
  if (offsets) std::memcpy(offsets, d.offsets.data(), std::min(range_cap, d.offsets.size()) * sizeof(int32_t));
  if (maps && !d.maps.empty()) std::memcpy(maps, d.maps.data(), std::min(map_cap, d.maps.size()));
  if (words) std::memcpy(words, d.words.data(), std::min(word_cap, d.words.size()) * sizeof(int32_t));
  return AR_OK;
}

void ar_schedule_free(ar_schedule* s) { delete reinterpret_cast<ar::Schedule*>(s); }

ar_status ar_schedule_info_get(const ar_schedule* sh, ar_schedule_info* info) {
  if (!sh || !info) return fail(AR_INVALID_ARGUMENT, "NULL argument");
  const ar::Schedule& s = *reinterpret_cast<const ar::Schedule*>(sh);
  info->steps = s.nsteps;
  info->slots = s.nslots;
  info->atoms = s.C;
  info->single_port = s.single_port ? 1 : 0;
  info->ops = int64_t(s.ops.size());
  info->finalize_ops = s.finalize_ops;
  info->fused_ok = s.fused_ok ? 1 : 0;
  info->ranges = int32_t(s.ranges.size());
  info->max_trees = s.max_trees;
  info->max_need = s.max_need;
  info->max_leaves = s.max_leaves;
  info->program_words = int32_t(s.prog.size());
  return AR_OK;
}

ar_status ar_schedule_export(const ar_schedule* sh, ar_oprec* ops, size_t cap, size_t* count) {
  if (!sh) return fail(AR_INVALID_ARGUMENT, "NULL schedule");
  const ar::Schedule& s = *reinterpret_cast<const ar::Schedule*>(sh);
  if (count) *count = s.ops.size();
  if (ops) std::memcpy(ops, s.ops.data(), std::min(cap, s.ops.size()) * sizeof(ar_oprec));
  return AR_OK;
}

ar_status ar_schedule_fused_export(const ar_schedule* sh, int64_t* starts, int64_t* lens, int32_t* offsets,
                                   size_t range_cap, int32_t* words, size_t word_cap, size_t* nranges,
                                   size_t* nwords) {
  if (!sh) return fail(AR_INVALID_ARGUMENT, "NULL schedule");
  const ar::Schedule& s = *reinterpret_cast<const ar::Schedule*>(sh);
  if (!s.fused_ok) return fail(AR_UNSUPPORTED, "no fused program: " + s.fused_error);
  if (nranges) *nranges = s.ranges.size();
  if (nwords) *nwords = s.prog.size();
  for (size_t r = 0; r < std::min(range_cap, s.ranges.size()); ++r) {
    if (starts) starts[r] = s.ranges[r].start;
    if (lens) lens[r] = s.ranges[r].len;
    if (offsets) offsets[r] = s.ranges[r].prog;
  }
  if (words) std::memcpy(words, s.prog.data(), std::min(word_cap, s.prog.size()) * sizeof(int32_t));
  return AR_OK;
}

ar_status ar_table_check(int32_t P, int64_t n, int32_t dtype, const ar_oprec* ops, size_t count,
                         int32_t* single_port) {
  if (!ops && count) return fail(AR_INVALID_ARGUMENT, "ops is NULL");
  if (dtype < AR_INT32 || dtype > AR_BF16) return fail(AR_INVALID_ARGUMENT, "unknown dtype");
  ar::TableCheck tc = ar::check_table(P, n, dtype, reinterpret_cast<const ar::OpRec*>(ops), count);
  if (single_port) *single_port = tc.single_port ? 1 : 0;
  if (!tc.ok) return fail(AR_INVALID_ARGUMENT, tc.message);
  return AR_OK;
}

ar_status ar_table_check_ex(const ar_call* call, const ar_oprec* ops, size_t count, int32_t* single_port) {
  if (!call) return fail(AR_INVALID_ARGUMENT, "call is NULL");
  if (!ops && count) return fail(AR_INVALID_ARGUMENT, "ops is NULL");
  if (call->dtype < AR_INT32 || call->dtype > AR_BF16) return fail(AR_INVALID_ARGUMENT, "unknown dtype");
  if (call->collective < AR_ALLREDUCE || call->collective > AR_ALL_GATHER)
    return fail(AR_INVALID_ARGUMENT, "unknown collective");
  if (call->n < 0) return fail(AR_INVALID_ARGUMENT, "n must be >= 0");
  ar::TableCheck tc = ar::check_table(call->P, call->n, call->dtype, reinterpret_cast<const ar::OpRec*>(ops),
                                      count, call->collective);
  if (single_port) *single_port = tc.single_port ? 1 : 0;
  if (!tc.ok) return fail(AR_INVALID_ARGUMENT, tc.message);
  return AR_OK;
}

ar_status ar_cost_report(const ar_schedule* sh, double alpha, double beta, double gamma, ar_cost* out) {
  if (!sh || !out) return fail(AR_INVALID_ARGUMENT, "NULL argument");
  const ar::Schedule& s = *reinterpret_cast<const ar::Schedule*>(sh);
  ar::CostOut c = ar::cost_walk(s, alpha, beta, gamma);
  out->steps = c.steps;
  out->sent_busiest = c.sent_busiest;
  out->recv_busiest = c.recv_busiest;
  out->reduced_busiest = c.reduced_busiest;
  out->sent_total = c.sent_total;
  out->reduced_total = c.reduced_total;
  out->max_rank_sent = c.max_rank_sent;
  out->max_rank_reduced = c.max_rank_reduced;
  out->predicted_seconds = c.predicted_seconds;
  out->closed_form_seconds = c.closed_form_seconds;
  out->literal_hbm_bytes = c.literal_hbm_bytes;
  out->fused_hbm_bytes = c.fused_hbm_bytes;
  out->essential_bytes = c.essential_bytes;
  return AR_OK;
}

ar_status ar_cost_steps(const ar_schedule* sh, int64_t* sent, int64_t* recv, int64_t* reduced) {
  if (!sh || !sent || !recv || !reduced) return fail(AR_INVALID_ARGUMENT, "NULL argument");
  ar::cost_steps(*reinterpret_cast<const ar::Schedule*>(sh), sent, recv, reduced);
  return AR_OK;
}

ar_status ar_grad_norm(const ar_grad* grads, int32_t count, const ar_clip* clip, void* stream) {
  return guarded([&] { return grad_call(grads, count, clip, false, stream, nullptr); });
}

ar_status ar_grad_clip(const ar_grad* grads, int32_t count, const ar_clip* clip, void* stream) {
  return guarded([&] { return grad_call(grads, count, clip, true, stream, nullptr); });
}

ar_status ar_grad_workspace_bytes(const ar_grad* grads, int32_t count, const ar_clip* clip, size_t* bytes) {
  if (!bytes) return fail(AR_INVALID_ARGUMENT, "bytes is NULL");
  // out plays no part in the size, known does: read the list as the clip does only if it asks for one
  return guarded([&] { return grad_call(grads, count, clip, clip && clip->known, nullptr, bytes); });
}

ar_status ar_allreduce_clip(void* const* bufs, const int64_t* n, int32_t buckets, int32_t P, int32_t dtype,
                            int32_t op, int32_t collective, const ar_clip* clip, void* stream) {
  return guarded([&] {
    ar::Clip c;
    ar::Buckets b;
    ar_status st = check_clip(clip, true, &c);
    if (st == AR_OK && c.known) st = fail(AR_INVALID_ARGUMENT, "known is for ar_grad_clip");
    if (st == AR_OK) st = check_buckets(bufs, true, n, buckets, P, dtype, op, collective, &b);
    if (st != AR_OK) return st;
    return finish(ar::run_allreduce_clip(b, c, stream));
  });
}

ar_status ar_allreduce_clip_workspace_bytes(const int64_t* n, int32_t buckets, int32_t P, int32_t dtype,
                                            int32_t op, int32_t collective, const ar_clip* clip, size_t* bytes) {
  if (!bytes) return fail(AR_INVALID_ARGUMENT, "bytes is NULL");
  return guarded([&] {
    ar::Clip c;
    ar::Buckets b;
    ar_status st = check_clip(clip, true, &c);
    if (st == AR_OK) st = check_buckets(nullptr, false, n, buckets, P, dtype, op, collective, &b);
    if (st != AR_OK) return st;
    *bytes = ar::allreduce_clip_workspace(b, c);
    return AR_OK;
  });
}

}  // extern "C"
