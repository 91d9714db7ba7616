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
