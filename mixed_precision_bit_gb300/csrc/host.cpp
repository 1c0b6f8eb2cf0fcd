// Host-side parts of the Kitty library: version, page sizes, effective bits and
// the physical page allocator (a PagedAttention-style free list of page ids).
#include <cmath>
#include <new>
#include <vector>

#include "host_common.h"
#include "kitty.h"

using kitty::blob_bytes;
using kitty::check_cfg;

struct kitty_alloc {
  int32_t num_pages;
  std::vector<int32_t> free_list;  // stack: back() is handed out next
  std::vector<uint8_t> in_use;
};

extern "C" int kitty_abi_version(void) { return 5; }

extern "C" int kitty_page_bytes(const kitty_cfg* cfg, size_t* per_head_blob, size_t* per_page) {
  const int rc = check_cfg(cfg);
  if (rc != KITTY_OK) return rc;
  const size_t b = blob_bytes(cfg->n_hi, cfg->lo_bit, kitty::v_bits(cfg));
  if (per_head_blob) *per_head_blob = b;
  if (per_page) *per_page = b * (size_t)cfg->num_kv_heads;
  return KITTY_OK;
}

// hi_fraction * hi_bit + (1 - hi_fraction) * lo_bit, hi_fraction = n_hi / D.
extern "C" float kitty_avg_bits(const kitty_cfg* cfg) {
  if (check_cfg(cfg) != KITTY_OK) return -1.0f;
  const double hf = (double)cfg->n_hi / cfg->head_dim;
  return (float)(hf * cfg->hi_bit + (1.0 - hf) * cfg->lo_bit);
}

extern "C" int kitty_alloc_create(int32_t num_pages, kitty_alloc** out) {
  if (num_pages < 0 || out == nullptr) return KITTY_ERR_INVALID_ARG;
  kitty_alloc* a = new (std::nothrow) kitty_alloc;
  if (a == nullptr) return KITTY_ERR_OOM;
  a->num_pages = num_pages;
  a->free_list.resize(num_pages);
  for (int32_t i = 0; i < num_pages; ++i) a->free_list[i] = num_pages - 1 - i;
  a->in_use.assign(num_pages, 0);
  *out = a;
  return KITTY_OK;
}

extern "C" int kitty_alloc_pages(kitty_alloc* a, int32_t n, int32_t* ids_out) {
  if (a == nullptr || n < 0 || (n > 0 && ids_out == nullptr)) return KITTY_ERR_INVALID_ARG;
  if ((size_t)n > a->free_list.size()) return KITTY_ERR_OOM;
  for (int32_t i = 0; i < n; ++i) {
    const int32_t id = a->free_list.back();
    a->free_list.pop_back();
    a->in_use[id] = 1;
    ids_out[i] = id;
  }
  return KITTY_OK;
}

extern "C" int kitty_free_pages(kitty_alloc* a, int32_t n, const int32_t* ids) {
  if (a == nullptr || n < 0 || (n > 0 && ids == nullptr)) return KITTY_ERR_INVALID_ARG;
  std::vector<uint8_t> seen(a->num_pages, 0);
  for (int32_t i = 0; i < n; ++i) {  // validate everything before changing anything
    const int32_t id = ids[i];
    if (id < 0 || id >= a->num_pages || !a->in_use[id] || seen[id]) return KITTY_ERR_INVALID_ARG;
    seen[id] = 1;
  }
  for (int32_t i = 0; i < n; ++i) {
    a->in_use[ids[i]] = 0;
    a->free_list.push_back(ids[i]);
  }
  return KITTY_OK;
}

extern "C" int32_t kitty_alloc_free_count(const kitty_alloc* a) {
  return a == nullptr ? -1 : (int32_t)a->free_list.size();
}

extern "C" void kitty_alloc_destroy(kitty_alloc* a) { delete a; }

// ---------------------------------------------------------------- rotation tables
namespace {
const double kTwoPi = 6.283185307179586476925286766559;
}

extern "C" int kitty_rope_frequencies(int32_t rot_dim, double base, const kitty_rope_scaling* sc,
                                      double* inv_freq, double* amplitude) {
  if (rot_dim <= 0 || rot_dim > 128 || rot_dim % 2 != 0 || !std::isfinite(base) || !(base > 1.0) ||
      inv_freq == nullptr || amplitude == nullptr)
    return KITTY_ERR_INVALID_ARG;
  const int kind = sc == nullptr ? KITTY_ROPE_PLAIN : sc->kind;
  if (kind < KITTY_ROPE_PLAIN || kind > KITTY_ROPE_BANDS) return KITTY_ERR_INVALID_ARG;
  if (kind != KITTY_ROPE_PLAIN && !(std::isfinite(sc->factor) && sc->factor >= 1.0))
    return KITTY_ERR_INVALID_ARG;
  const bool bands = kind == KITTY_ROPE_YARN || kind == KITTY_ROPE_BANDS;
  if (bands && !(sc->trained >= 1 && std::isfinite(sc->fast) && sc->slow > 0.0 && sc->fast > sc->slow))
    return KITTY_ERR_INVALID_ARG;
  if (kind == KITTY_ROPE_NTK) {
    if (rot_dim == 2) return KITTY_ERR_INVALID_ARG;
    base *= std::pow(sc->factor, (double)rot_dim / (rot_dim - 2));
  }
  double low = 0.0, high = 0.0;  // YaRN: the ramp over pair indices
  if (kind == KITTY_ROPE_YARN) {
    auto pair_of = [&](double n) {
      return rot_dim * std::log(sc->trained / (kTwoPi * n)) / (2.0 * std::log(base));
    };
    low = std::fmax(std::floor(pair_of(sc->fast)), 0.0);
    high = std::fmin(std::ceil(pair_of(sc->slow)), rot_dim - 1.0);
    if (!(high > low)) high = low + 0.001;  // a step instead of a ramp
  }
  for (int j = 0; j < rot_dim / 2; ++j) {
    double f = std::pow(base, -2.0 * j / rot_dim);
    if (kind == KITTY_ROPE_LINEAR) {
      f /= sc->factor;
    } else if (kind == KITTY_ROPE_YARN) {
      const double u = std::fmin(std::fmax((j - low) / (high - low), 0.0), 1.0);
      f = f * (1.0 - u) + f / sc->factor * u;
    } else if (kind == KITTY_ROPE_BANDS) {
      const double turns = sc->trained * f / kTwoPi;  // over the trained length
      const double u = std::fmin(std::fmax((turns - sc->slow) / (sc->fast - sc->slow), 0.0), 1.0);
      f = f / sc->factor * (1.0 - u) + f * u;
    }
    inv_freq[j] = f;
  }
  *amplitude = kind == KITTY_ROPE_YARN ? 0.1 * std::log(sc->factor) + 1.0 : 1.0;
  return KITTY_OK;
}

extern "C" int kitty_rope_turns(const double* inv_freq, int32_t n, uint64_t* turns) {
  if (n < 0 || (n > 0 && (inv_freq == nullptr || turns == nullptr))) return KITTY_ERR_INVALID_ARG;
  for (int32_t j = 0; j < n; ++j)
    if (!std::isfinite(inv_freq[j])) return KITTY_ERR_INVALID_ARG;
  for (int32_t j = 0; j < n; ++j) {
    // the magnitude's fraction of a turn in [0, 1) (exact), in two 32-bit pieces (both
    // products are exact); a negative frequency is its negative modulo 2^64
    double x = std::fabs(inv_freq[j] / kTwoPi);
    x -= std::floor(x);
    const double hi = std::floor(x * 4294967296.0);
    const double lo = std::floor((x * 4294967296.0 - hi) * 4294967296.0);
    const uint64_t t = ((uint64_t)hi << 32) + (uint64_t)lo;
    turns[j] = inv_freq[j] < 0.0 ? 0 - t : t;
  }
  return KITTY_OK;
}
