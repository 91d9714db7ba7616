// Python side of the 8-bit cache, the reading of rows and the attention with modified scores: a part of binding.cpp, whose
// helpers it uses (included there, inside its namespace).

// block_tables, cu_q_lens, positions, held_lens, k_new, v_new, stream
PyObject* append_int8(Pool* p, Args a) {
  const Batch b(p, a[0], a[1], "cu_q_lens");
  const int64_t T = tensor(a[2], "positions", 1).size(0);
  const int32_t* pos = address<int32_t>(p, a[2], "positions", at::kInt, {T});
  const int32_t* held = address<int32_t>(p, a[3], "held_lens", at::kInt, {b.reqs});
  const void* k = address(p, a[4], "k_new", at::kBFloat16, {T, p->num_kv_heads, p->head_dim});
  const void* v = address(p, a[5], "v_new", at::kBFloat16, {T, p->num_kv_heads, p->head_dim});
  const Call call(p, a[6]);
  run(pkv_append_int8, p->handle, b.tables, count(b.width), count(b.reqs), b.cu, pos, held, k, v, count(T), call.stream());
  Py_RETURN_NONE;
}

// block_tables, cu_lens, positions, k_out, v_out, stream
PyObject* read_rows(Pool* p, Args a) {
  const Batch b(p, a[0], a[1], "cu_lens");
  const int64_t T = tensor(a[2], "positions", 1).size(0);
  const int32_t* pos = address<int32_t>(p, a[2], "positions", at::kInt, {T});
  const Call call(p, a[5]);
  Table k(p, call, a[3], "k_out", {T, p->num_kv_heads, p->head_dim}, at::kBFloat16);
  Table v(p, call, a[4], "v_out", {T, p->num_kv_heads, p->head_dim}, at::kBFloat16);
  run(pkv_read_rows, p->handle, b.tables, count(b.width), count(b.reqs), b.cu, pos, count(T), k.data, v.data, call.stream());
  PyObject *x = k.result(), *y = v.result(), *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// q, q_positions, block_tables, ctx_lens, cu_q_lens, scale, softcap, window, slopes, first_keys, prefix_lens, out, lse,
// workspace, stream, want_lse
PyObject* score_attn(Pool* p, Args a) {
  const Batch b(p, a[2], a[4], "cu_q_lens");
  const Query q(p, a[0]);
  const int32_t* pos = address<int32_t>(p, a[1], "q_positions", at::kInt, {q.tokens});
  const int32_t* ctx = address<int32_t>(p, a[3], "ctx_lens", at::kInt, {b.reqs});
  const float scale = number(a[5]);
  pkv_score_desc d{number(a[6]), integer(a[7]), nullptr, nullptr, nullptr};
  if (a[8] != Py_None) d.slopes = address<float>(p, a[8], "slopes", at::kFloat, {q.heads});
  if (a[9] != Py_None) d.first_keys = address<int32_t>(p, a[9], "first_keys", at::kInt, {q.tokens});
  if (a[10] != Py_None) d.prefix_lens = address<int32_t>(p, a[10], "prefix_lens", at::kInt, {b.reqs});
  Call call(p, a[14]);
  Output out(p, call, q, a[11], a[12], a[15] == Py_True);
  size_t size = 0;
  check(pkv_score_attn_workspace_size(p->handle, count(q.heads), count(b.width), count(b.reqs), count(q.tokens), &size));
  const at::Tensor ws = call.workspace(a[13], size);
  run(pkv_score_attn, p->handle, q.q, count(q.heads), pos, b.tables, count(b.width), ctx, b.cu, count(b.reqs),
      count(q.tokens), static_cast<const pkv_score_desc*>(&d), scale, out.o, out.lse, ws.data_ptr(),
      static_cast<size_t>(ws.numel()), call.stream());
  return out.result();
}
